"""Long sums of the expert layer (sar_expert_layer) over values of one sign, whose errors do not cancel: no chain of the
tensor cores' cut-off additions runs over all of k.

Bounds, relative, for terms of one sign: a chain has at most 128 products whose sums are off by up to two units in the last
place (4 U) each, 512 U; the chains are added rounded to nearest, U each: on the way out one for every 512 of k, on the way
in, whose k four warps share, one for every 4096, and 64 more at most for the shares; operands in two numbers leave 2^-16 at
most (bf16, as tests/block_ref.py) or 16 U."""
import pytest
import torch

from tests import operator_ref as ref
from tests.test_gpu_expert_layer import layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


def bound(joins, dtype):
    return ref.SLACK * ((512 + joins + 64 + 16) * ref.U + (2.0 ** -16 if dtype == "bf16" else 0.0))


def positive(tokens, cols, hidden, dtype, seed, x_size=1.0, in_size=1.0, out_size=1.0):
    """Inputs above zero for one expert; the tokens' sizes are spread evenly over a factor of two, so that the outputs'
    roundings are as well."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = ref.DTYPES[dtype]

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")
    x = (x_size * rand(tokens, cols) * 2 ** rand(tokens, 1)).to(d)
    w_in, w_out = (in_size * rand(1, hidden, cols)).to(d), (out_size * rand(1, cols, hidden)).to(d)
    return x, torch.zeros(tokens, 1, dtype=torch.int32, device="cuda"), w_in, w_out


def relative(got, x, w_in, w_out):
    want = (x.double() @ w_in[0].double().T) @ w_out[0].double().T
    return got.double() / want - 1


def check(rel, joins, dtype):
    unit = ref.OUT[ref.DTYPES[dtype]]
    assert rel.abs().max() <= bound(joins, dtype) + unit, rel.abs().max().item()
    # the outputs' own roundings are independent and up to `unit` each: six standard deviations of their mean
    assert abs(rel.mean().item()) <= bound(joins, dtype) + 6 * unit / 3 ** 0.5 / rel.numel() ** 0.5, rel.mean().item()


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("tokens,hidden,cols", [(1024, 65536, 16), (1024, 65535, 16), (600, 40000, 33), (90, 131072, 24)])
def test_long_way_out(sar, tokens, hidden, cols, dtype):
    """h is about 4, the output 2^-3 of hidden's size: inside binary16's range, its weights normal numbers."""
    x, ids, w_in, w_out = positive(tokens, cols, hidden, dtype, seed=hidden, out_size=2.0 ** -9)
    check(relative(layer(sar, x, ids, w_in, w_out, None, "relu"), x, w_in, w_out), hidden / 512, dtype)


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("tokens,cols", [(8, 2 ** 20), (3, 2 ** 20 - 5), (40, 500001)])
def test_long_way_in(sar, tokens, cols, dtype):
    x, ids, w_in, w_out = positive(tokens, cols, 16, dtype, seed=cols, x_size=2.0 ** -8, in_size=2.0 ** -8)
    check(relative(layer(sar, x, ids, w_in, w_out, None, "relu"), x, w_in, w_out), cols / 4096, dtype)


@pytest.mark.parametrize("value", [0.6864250, 0.9828040, 1.8147260, 1.4707840])
def test_equal_terms_in_binary32(sar, value):
    """Additions of one term again and again err to one side within a power of two: 16384 in a row by up to 2e-4."""
    cols = 2 ** 20
    x, ids = torch.full((8, cols), value, device="cuda"), torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    w_in, w_out = torch.full((1, 16, cols), value, device="cuda"), torch.full((1, cols, 16), value, device="cuda")
    got = layer(sar, x, ids, w_in, w_out, None, "relu")
    check(relative(got, x, w_in, w_out), cols / 4096, "fp32")
