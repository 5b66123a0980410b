"""The bounded wait between the blocks of a cluster (the gated recurrence's exchange) without a GPU fault: two blocks
expect each other's sums, neither sends them, both give up after about 2^20 cycles, and the host reads it as
GDN_ERR_TIMEOUT; the context stays usable."""
import pytest
import torch


@pytest.mark.gpu
def test_expired_cluster_wait_is_reported_and_the_context_survives(cuda_lib):
    from test_glr import check
    cuda_lib.gdn_device_status()  # start from a clean error word
    for limit in (1 << 20, 0):
        cuda_lib.gdn_selftest_expired_cluster_wait(limit)
        with pytest.raises(cuda_lib.GdnError) as e:
            cuda_lib.gdn_device_status()
        assert e.value.status == 4  # GDN_ERR_TIMEOUT
        cuda_lib.gdn_device_status()  # the word was read and cleared
    # rounds of a cluster's blocks are right behind it, and none of their waits expires
    check(cuda_lib, (1605,), False, 64, torch.float32, "log", None, True)
    torch.cuda.synchronize()
    cuda_lib.gdn_device_status()


def test_selftest_rejects_a_bad_limit_without_a_device():
    from linear_attention_prefill_gb300 import _build, binding
    _build.build()
    lib = binding.load_library()
    assert lib.gdn_selftest_expired_cluster_wait(-1, None) == 1
    assert lib.gdn_selftest_expired_cluster_wait(1 << 40, None) == 1
