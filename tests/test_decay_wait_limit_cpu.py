"""The wait limit of the bf16 decay kernels is a setting of the calling thread."""
import os
import threading

import pytest

from linear_attention_recurrence_07_b200 import binding


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIBRARY_PATH):
        from linear_attention_recurrence_07_b200 import build
        build.build()
    return binding.library()


def test_the_limit_is_set_and_restored(lib):
    assert lib.gdn_get_decay_wait_limit() == 0
    with binding.decay_wait_limit(1 << 40):
        assert lib.gdn_get_decay_wait_limit() == 1 << 40
        with binding.decay_wait_limit(0):
            assert lib.gdn_get_decay_wait_limit() == 0
        assert lib.gdn_get_decay_wait_limit() == 1 << 40
    assert lib.gdn_get_decay_wait_limit() == 0


def test_a_negative_limit_is_refused(lib):
    assert lib.gdn_set_decay_wait_limit(-1) == binding.GDN_ERR_INVALID_ARG
    with pytest.raises(binding.GdnError, match="INVALID_ARG"):
        with binding.decay_wait_limit(-5):
            pass
    assert lib.gdn_get_decay_wait_limit() == 0


def test_other_threads_keep_their_own(lib):
    seen = []
    with binding.decay_wait_limit(123):
        t = threading.Thread(target=lambda: seen.append(lib.gdn_get_decay_wait_limit()))
        t.start()
        t.join()
    assert seen == [0]
