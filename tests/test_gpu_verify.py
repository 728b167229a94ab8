"""gdn_verify against its definition in float64 (tests/draft_ref.py): whole numbers, so the
results are equal. The sums of both are float64 in different orders: they agree to about
V * 2^-53, so a draw that lands within that of a token's border could differ; the seeds here
are fixed and no draw does."""
import numpy as np
import pytest
import torch

from gated_delta_rule_depthwise_amd import binding as G
from gated_delta_rule_depthwise_amd.runner import verify
from tests import draft_ref

pytestmark = pytest.mark.gpu


def make(B, T, V, seed, dtype=torch.float32, noise=0.7):
    gen = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, T + 1, V, generator=gen) * 2
    p = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits[:, :T] + noise * torch.randn(B, T, V, generator=gen), -1).to(dtype)
    tok = torch.multinomial(q.reshape(-1, V).float(), 1, generator=gen).view(B, T).to(torch.int32) if T else \
        torch.zeros(B, 0, dtype=torch.int32)
    return p.cuda(), q.cuda(), tok.cuda(), torch.rand(B, T + 1, generator=gen).cuda()


def check(p, tok, u, q=None, num=None):
    length = torch.arange(p.shape[0], dtype=torch.int32, device="cuda")
    rc, acc, nxt = verify(p, tok, u, draft=q, num=num, len=length)
    torch.cuda.synchronize()
    assert rc == 0
    ra, rn = draft_ref.verify(p, tok, u, draft=q, num=num)
    assert acc.tolist() == ra.tolist()
    assert nxt.tolist() == rn.tolist()
    assert length.tolist() == [b + a + 1 for b, a in enumerate(ra.tolist())]
    return ra, rn


@pytest.mark.parametrize("V", [1, 2, 63, 64, 257, 4095, 4096, 4097, 50257, 300001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_vocabularies(V, dtype):
    p, q, tok, u = make(7, 3, V, 100 + V, dtype)
    check(p, tok, u, q)
    check(p, tok, u)                                            # drafts without probabilities


@pytest.mark.parametrize("B,T", [(1, 0), (5, 0), (1, 1), (130, 2), (3, 17), (2, 300)])
def test_draft_counts(B, T):
    p, q, tok, u = make(B, T, 301, 7 + T, noise=0.05)
    a, _ = check(p, tok, u, q if T else None)
    if T == 300:
        assert a.max() > 8
    num = torch.arange(B, dtype=torch.int32, device="cuda") % (T + 2) - 1     # -1 .. T
    check(p, tok, u, q if T else None, num=num)
    num.fill_(T + 5)
    check(p, tok, u, q if T else None, num=num)


@pytest.mark.parametrize("V", [1000, 9000, 40000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_borders(dtype, V):
    """The random numbers' ends, a proposal equal to the target (nothing is left over), rows
    without weight, and weights that are NaN, negative or infinite."""
    p, q, tok, u = make(6, 2, V, 9, dtype)
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    q[2] = p[2, :2]
    tok[2] = p[2, :2].float().argmax(-1).to(torch.int32)
    u[2, 0] = 1 - 2.0 ** -24                                    # still below p / q = 1
    q[3, 0] = (p[3, 0].float() * 2).to(dtype)                   # p <= q everywhere: drawn from p
    u[3, 0] = 0.99
    p[4] = 0.0                                                  # no token at all
    p[5, 0, ::3], p[5, 0, 1::3] = float("nan"), -1.0
    tok[5, 0] = 3                                               # NaN: refused
    a, n = check(p, tok, u, q)
    assert a[2] == 2 and a[3] == 0 and n[4] == -1 and a[5] == 0 and n[5] % 3 == 2
    check(p, tok, u)


def test_a_batch_of_long_rows():
    """Rows of more than one part in a batch that takes one workgroup each."""
    p, q, tok, u = make(130, 1, 40001, 19, torch.bfloat16)
    check(p, tok, u, q)


def test_weight_in_one_place():
    """All the weight on the first, the last, or a token in the middle of a part."""
    for V, at in ((9000, 0), (9000, 1), (9000, 4095), (9000, 4096), (9000, 8999), (7, 6), (8192, 8191),
                  (8193, 8192), (40000, 8191), (40000, 8192), (40000, 39999)):
        p = torch.zeros(2, 1, V, device="cuda")
        p[:, 0, at] = 0.25
        u = torch.tensor([[0.0], [1 - 2.0 ** -24]], device="cuda")
        _, n = check(p, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), u)
        assert n.tolist() == [at, at]


def test_tokens_outside_the_vocabulary():
    p, q, tok, u = make(4, 2, 65, 11)
    tok[0, 0], tok[1, 0], tok[2, 1], tok[3, 1] = -1, 65, 2147483647, -2147483648
    u[:, 0] = torch.tensor([0.0, 0.0, 0.0, 0.0])
    check(p, tok, u, q)
    check(p, tok, u)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off,ld", [(1, 5003), (3, 5001), (0, 5008)])
def test_strides_and_alignment(dtype, off, ld):
    """Rows of any stride, starting at any element; what lies between them is not read."""
    B, T, V = 3, 2, 4999
    p, q, tok, u = make(B, T, V, 13, dtype)
    ra, rn = check(p, tok, u, q)
    bp = torch.full((off + B * (T + 1) * ld,), float("nan"), dtype=dtype, device="cuda")
    bq = torch.full((off + 2 + B * T * ld,), float("nan"), dtype=dtype, device="cuda")
    wp = torch.as_strided(bp, (B * (T + 1), V), (ld, 1), off)
    wq = torch.as_strided(bq, (B * T, V), (ld, 1), off + 2)
    wp.copy_(p.view(-1, V))
    wq.copy_(q.view(-1, V))
    n = G.gdn_verify_workspace_bytes(B, T, V)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    acc, nxt = torch.zeros(2, B, dtype=torch.int32, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert G.gdn_verify(wp, ld, wq, ld, G.GDN_BF16 if dtype == torch.bfloat16 else G.GDN_F32, tok, None, u, B, T,
                        V, acc, nxt, None, ws, n, s) == 0
    torch.cuda.synchronize()
    assert acc.tolist() == ra.tolist() and nxt.tolist() == rn.tolist()


def test_rows_past_32_bits():
    """Row offsets past 2^31 elements."""
    B, T, V, ld = 2, 1, 300, (1 << 30) // 2 + 64
    p, q, tok, u = make(B, T, V, 17, torch.bfloat16)
    ra, rn = check(p, tok, u, q)
    big = torch.zeros(4 * ld, dtype=torch.bfloat16, device="cuda")
    torch.as_strided(big, (4, V), (ld, 1), 0).copy_(p.view(-1, V))
    assert 3 * ld * 2 > 2 ** 31
    n = G.gdn_verify_workspace_bytes(B, T, V)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    acc, nxt = torch.zeros(2, B, dtype=torch.int32, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert G.gdn_verify(big, ld, q, V, G.GDN_BF16, tok, None, u, B, T, V, acc, nxt, None, ws, n, s) == 0
    torch.cuda.synchronize()
    assert acc.tolist() == ra.tolist() and nxt.tolist() == rn.tolist()


def test_draws_follow_the_target():
    """Speculative sampling keeps the target's distribution: the first token of 20000 streams
    with one draft each. Each count is binomial: 6 standard deviations of B p (1 - p)."""
    B, V = 20000, 5
    gen = torch.Generator(device="cuda").manual_seed(3)
    p1 = torch.tensor([0.4, 0.3, 0.15, 0.1, 0.05], device="cuda")
    q1 = torch.tensor([0.1, 0.5, 0.2, 0.1, 0.1], device="cuda")
    tok = torch.multinomial(q1.expand(B, V), 1, generator=gen).to(torch.int32)
    u = torch.rand(B, 2, generator=gen, device="cuda")
    rc, acc, nxt = verify(p1.expand(B, 2, V).contiguous(), tok, u, draft=q1.expand(B, 1, V).contiguous())
    assert rc == 0
    first = torch.where(acc > 0, tok[:, 0], nxt).long()
    got = np.bincount(first.cpu().numpy(), minlength=V)
    p = p1.double().cpu().numpy()
    assert np.all(np.abs(got - B * p) <= 6 * np.sqrt(B * p * (1 - p)))
