"""Numbers that the training operators' binding is given and that a C integer
cannot hold (CPU only): refused, not taken modulo 2^32 or 2^64."""
import pytest
import torch

from row_wise_rmsnorm_fwd_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("kw", [
    dict(max_distance=(1 << 32) + 128), dict(max_distance=128 - (1 << 32)),
    dict(q_offset=1 << 64), dict(q_offset=-(1 << 63) - 1), dict(q_offset=(1 << 65) + 7)])
def test_rule_numbers_past_the_c_types(kw):
    x, table = torch.zeros((2, 3, 4, 5)), torch.zeros((32, 3))
    name = next(iter(kw))
    with pytest.raises(ValueError, match=name):
        binding.rowsoftmax_relbias_fwd_f32(x, table, **kw)
    with pytest.raises(ValueError, match=name):
        binding.rowsoftmax_relbias_bwd_f32(x, x, 32, **kw)


def test_bucket_numbers_past_the_c_types():
    with pytest.raises(ValueError, match="num_buckets"):
        binding.rowsoftmax_relbias_bwd_f32(torch.zeros((2, 3, 4, 5)), torch.zeros((2, 3, 4, 5)),
                                           (1 << 32) + 32)
    with pytest.raises(ValueError, match="num_buckets"):
        binding.rowsoftmax_relbias_bucket(0, (1 << 32) + 32)
    with pytest.raises(ValueError, match="max_distance"):
        binding.rowsoftmax_relbias_bucket(0, 32, (1 << 32) + 128)
    for r in (1 << 63, (1 << 64) + 5, -(1 << 63) - 1):
        with pytest.raises(ValueError, match="relative"):
            binding.rowsoftmax_relbias_bucket(r, 32)
    assert binding.rowsoftmax_relbias_bucket((1 << 63) - 1, 32) == 31
    assert binding.rowsoftmax_relbias_bucket(0, 31) == -1
