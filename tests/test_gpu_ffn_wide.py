"""Very many outputs of few tokens: launches of the direct kernels would pass
2^32 threads, and the runtime counts them in 32 bits."""
import pytest
import torch

import message_allreduce_amd as llar

pytestmark = pytest.mark.gpu

K = 8


def ones_and_twos(rows, seed):
    """Values whose sums of products are exact in every type: +-1, +-2."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.randint(1, 3, (rows, K), generator=g, device="cuda", dtype=torch.int8)
    t *= torch.randint(0, 2, (rows, K), generator=g, device="cuda", dtype=torch.int8) * 2 - 1
    return t.bfloat16()


def same(got, want):
    """Compares in pieces: the whole in another type would be large."""
    piece = 1 << 22
    for at in range(0, got.shape[1], piece):
        assert torch.equal(got[:, at:at + piece], want(at, min(at + piece, got.shape[1]))), at


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("m,n", [(1, (1 << 27) + 24), (2, (1 << 25) + 24), (3, (1 << 26) + 24)])
def test_linear(m, n, layout):
    if layout == "col":
        n = min(n, (1 << 21) - 8)  # a contiguous axis is no longer
    x, w = ones_and_twos(m, 1), ones_and_twos(n, 2)
    wo = w if layout == "row" else w.t().contiguous().t()
    same(llar.linear(x, wo), lambda a, b: (x.float() @ w[a:b].float().t()).bfloat16())


@pytest.mark.parametrize("m,n", [(1, (1 << 26) + 24), (3, (1 << 25) + 24)])
def test_gated(m, n):
    x, wg, wu = ones_and_twos(m, 1), ones_and_twos(n, 2), ones_and_twos(n, 3)

    def want(a, b):
        g, u = (x.float() @ w[a:b].float().t() for w in (wg, wu))
        return (torch.relu(g) * u).bfloat16()
    same(llar.gated_ffn(x, wg, wu, activation="relu"), want)


def test_a_pass_beyond_the_limit_is_refused():
    """A copy of 2^24 rows of 2049, at 8 elements a thread, would take more than 2^32 threads."""
    x = torch.ones(1, 2049, dtype=torch.bfloat16, device="cuda").expand(1 << 24, 2049)
    with pytest.raises(llar.LlarError):
        llar.linear(x, torch.ones(1, 2049, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.empty_cache()
