"""GPU parity of the layer operators (gdn_layer.h) against their float64 definitions (oracle.layer).

Tolerances, all relative to the largest value of the compared array:
  fp32 outputs of fp32 arithmetic: a sum of n products rounds to about sqrt(n) 2^-24 and the
    recurrence adds a few hundred such steps: 2^-15 holds with a wide margin.
  states of the tensor-core kernel: operands enter as pairs of bf16 (2^-17 of each entry), about
    six such roundings: 2^-14.
  bf16 outputs: 2^-9 for the rounding itself and 2^-9 of each term for the bf16 operands of the
    output products, whose sum may cancel: 2^-6.
  norms and gates in bf16 are rounded once: 2^-8 of each value.
"""
import numpy as np
import pytest
import torch

from gated_delta_net_gb300 import binding as gb
from oracle import layer as OL

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2.0 ** -15, torch.bfloat16: 2.0 ** -6}
TOL_STATE = {torch.float32: 2.0 ** -15, torch.bfloat16: 2.0 ** -14}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_net_gb300 import build
    build.build()
    gb.lib()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def close(got, ref, tol):
    got = f64(got)
    assert got.shape == ref.shape
    assert np.all(np.isfinite(got))
    if ref.size:
        assert np.max(np.abs(got - ref)) <= tol * max(np.max(np.abs(ref)), 1e-30)


def offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def tokens(seed, T, hk, hv, dk, dv, dtype, slow=False):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    unit = torch.nn.functional.normalize
    q, k = unit(n(T, hk, dk), dim=-1).to(dtype).cuda(), unit(n(T, hk, dk), dim=-1).to(dtype).cuda()
    v = n(T, hv, dv).to(dtype).cuda()
    g = -(0.02 if slow else 1.0) * torch.nn.functional.softplus(n(T, hv))
    return q, k, v, g.float().cuda(), torch.sigmoid(n(T, hv)).float().cuda()


def pool(seed, n, hv, dk, dv):
    gen = torch.Generator().manual_seed(seed)
    return (0.1 * torch.randn(n, hv, dv, dk, generator=gen)).cuda()


LENGTHS = [[1], [2], [63], [64], [65], [128], [0, 1, 0], [1, 64, 0, 17, 130], [200, 3], [331]]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_prefill_lengths(lengths, dtype):
    T, hk, hv = sum(lengths), 1, 2
    x = tokens(T, T, hk, hv, 128, 128, dtype, slow=True)
    off = offsets(lengths)
    S0 = pool(1, len(lengths), hv, 128, 128)
    st = gb.new_status()
    o, S = gb.gdn_prefill(*x, off, max(lengths), S0=S0, scale=0.25, dev_status=st)
    gb.check_status(st)
    ro, rS = OL.prefill(*map(f64, x), off.cpu().numpy(), S0=f64(S0), scale=0.25)
    close(o, ro, TOL[dtype])
    close(S, rS, TOL_STATE[dtype])
    assert np.array_equal(f64(S0), f64(pool(1, len(lengths), hv, 128, 128)))  # only read


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 1, 16, 16), (2, 4, 32, 128), (1, 3, 64, 64), (2, 2, 128, 16), (1, 2, 16, 128),
                                         (2, 4, 128, 128), (1, 4, 128, 128), (1, 2, 128, 64)])
def test_prefill_widths_and_types(hk, hv, dk, dv, dtype, out_dtype):
    lengths = [70, 5, 129]
    x = tokens(5, sum(lengths), hk, hv, dk, dv, dtype)
    off = offsets(lengths)
    st = gb.new_status()
    o, S = gb.gdn_prefill(*x, off, 129, scale=dk ** -0.5, out_dtype=out_dtype, dev_status=st)
    gb.check_status(st)
    assert o.dtype == out_dtype
    ro, rS = OL.prefill(*map(f64, x), off.cpu().numpy(), scale=dk ** -0.5)
    close(o, ro, TOL[BF if BF in (dtype, out_dtype) else F32])
    close(S, rS, TOL_STATE[dtype])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_prefill_strided_tokens_slots_fresh_in_place(dtype, pad):
    lengths, hk, hv, d, n = [80, 0, 33, 150], 2, 4, 128, 7
    T = sum(lengths)
    q, k, v, g, beta = tokens(8, T, hk, hv, d, d, dtype)
    rows = torch.full((T, (2 * hk + hv) * d + pad), float("nan"), dtype=dtype, device="cuda")
    qs = rows[:, :hk * d].view(T, hk, d)
    ks = rows[:, hk * d:2 * hk * d].view(T, hk, d)
    vs = rows[:, 2 * hk * d:(2 * hk + hv) * d].view(T, hv, d)
    qs.copy_(q), ks.copy_(k), vs.copy_(v)
    S = pool(2, n, hv, d, d)
    before = f64(S)
    slots = torch.tensor([5, 0, 3, 1], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([0, 0, 1, 0], dtype=torch.int32, device="cuda")
    off = offsets(lengths)
    st = gb.new_status()
    o, S2 = gb.gdn_prefill(qs, ks, vs, g, beta, off, 150, S0=S, S_new=S, slots=slots, fresh=fresh, dev_status=st)
    gb.check_status(st)
    assert S2 is S
    ro, rS = OL.prefill(*map(f64, (q, k, v, g, beta)), off.cpu().numpy(), S0=before, slots=slots.cpu().numpy(),
                        fresh=fresh.cpu().numpy())
    close(o, ro, TOL[dtype])
    close(S, rS, TOL_STATE[dtype])
    for s in (2, 4, 6, 0):
        assert np.array_equal(f64(S)[s], before[s])


@pytest.mark.parametrize("hv,length", [(1, 1000), (2, 2500), (1, 4096)])
def test_prefill_long_prompt_many_segments(hv, length):
    x = tokens(11, length, 1, hv, 128, 128, BF, slow=True)
    off = offsets([length])
    S0 = pool(3, 1, hv, 128, 128)
    st = gb.new_status()
    o, S = gb.gdn_prefill(*x, off, length, S0=S0, dev_status=st)
    gb.check_status(st)
    ro, rS = OL.prefill(*map(f64, x), [0, length], S0=f64(S0))
    close(o, ro, TOL[BF])
    close(S, rS, TOL_STATE[BF])


def test_prefill_segments_in_place():
    # prompts of several segments and of one, states in their pool's places, some of them not read
    lengths, hv, n = [700, 64, 0, 2000, 129], 2, 6
    x = tokens(19, sum(lengths), 1, hv, 128, 128, BF, slow=True)
    off = offsets(lengths)
    S = pool(8, n, hv, 128, 128)
    before = f64(S)
    slots = torch.tensor([4, 1, 0, 3, 5], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([0, 0, 0, 0, 1], dtype=torch.int32, device="cuda")
    assert gb.gdn_prefill_workspace(5, 1, hv, 128, 128, sum(lengths), 2000) > 0
    ro, rS = OL.prefill(*map(f64, x), off.cpu().numpy(), S0=before, slots=slots.cpu().numpy(), fresh=fresh.cpu().numpy())
    for _ in range(3):
        S.copy_(torch.from_numpy(before).float())
        st = gb.new_status()
        o, _ = gb.gdn_prefill(*x, off, 2000, S0=S, S_new=S, slots=slots, fresh=fresh, dev_status=st)
        gb.check_status(st)
        close(o, ro, TOL[BF])
        close(S, rS, TOL_STATE[BF])
    assert np.array_equal(f64(S)[2], before[2])
    with pytest.raises(gb.GdnError):
        gb.gdn_prefill(*x, off, 2000, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_prefill_correlated_unnormalised_keys():
    # neighbouring keys almost alike and longer than one: the chunk's system is far from the identity
    T = 192
    q, k, v, g, beta = tokens(12, T, 1, 2, 128, 128, BF, slow=True)
    k = (0.9 * k[:1].float() + 0.45 * k.float()).to(BF)
    off = offsets([T])
    o, S = gb.gdn_prefill(q, k, v, g, beta, off, T)
    ro, rS = OL.prefill(*map(f64, (q, k, v, g, beta)), [0, T])
    close(o, ro, TOL[BF])
    close(S, rS, TOL_STATE[BF])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prefill_extreme_decays(dtype):
    # tokens that forget everything, tokens that forget nothing, large decays before slow ones
    T = 150
    q, k, v, g, beta = tokens(13, T, 1, 2, 128, 128, dtype, slow=True)
    g[10] = -float("inf")
    g[11] = -float("inf")
    g[70] = -3.0e38
    g[90] = -60.0
    g[100:110] = 0.0
    beta[120:130] = 0.0
    off = offsets([T])
    S0 = pool(4, 1, 2, 128, 128)
    o, S = gb.gdn_prefill(q, k, v, g, beta, off, T, S0=S0)
    ro, rS = OL.prefill(*map(f64, (q, k, v, g, beta)), [0, T], S0=f64(S0))
    close(o, ro, TOL[dtype])
    close(S, rS, TOL_STATE[dtype])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prefill_does_not_read_its_neighbours(dtype):
    # the prompts before and after, and an unread state, are full of NaN
    lengths = [70, 100, 90]
    q, k, v, g, beta = tokens(14, 260, 1, 2, 128, 128, dtype)
    ref = [t[70:170].clone() for t in (q, k, v, g, beta)]
    for t in (q, k, v, g, beta):
        t[:70] = float("nan")
        t[170:] = float("nan")
    S0 = torch.full((3, 2, 128, 128), float("nan"), device="cuda")
    fresh = torch.ones(3, dtype=torch.int32, device="cuda")
    o, S = gb.gdn_prefill(q, k, v, g, beta, offsets(lengths), 100, S0=S0, fresh=fresh)
    ro, rS = OL.prefill(*map(f64, ref), [0, 100])
    close(o[70:170], ro, TOL[dtype])
    close(S[1:2], rS, TOL_STATE[dtype])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prefill_skips_bad_requests(dtype):
    lengths = [70, 100, 90, 64]
    x = tokens(15, 324, 1, 2, 128, 128, dtype)
    for kw, bit in ((dict(max_tokens=90), 4), (dict(slots=[0, 4, 2, 3]), 128), (dict(slots=[0, -1, 2, 3]), 128),
                    (dict(off=[0, 70, 60, 260, 324]), 32), (dict(off=[0, 70, 170, 260, 325]), 32)):
        st = gb.new_status()
        out = torch.full((324, 2, 128), 7.0, dtype=dtype, device="cuda")
        S = torch.full((4, 2, 128, 128), 7.0, device="cuda")
        off = torch.tensor(kw["off"], dtype=torch.int32, device="cuda") if "off" in kw else offsets(lengths)
        slots = torch.tensor(kw["slots"], dtype=torch.int32, device="cuda") if "slots" in kw else None
        gb.gdn_prefill(*x, off, kw.get("max_tokens", 200), slots=slots, out=out, S_new=S, dev_status=st)
        assert int(st.item()) & bit, kw
        bad = 3 if kw.get("off", [0])[-1] == 325 else 1
        assert bool((S[bad] == 7.0).all())
        ro, rS = OL.prefill(*[f64(t)[:70] for t in x], [0, 70])
        close(out[:60], ro[:60], TOL[dtype])  # rows 60 to 70 belong to two requests where the offsets descend
        close(S[:1], rS, TOL_STATE[dtype])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prefill_skips_offsets_at_the_ends_of_their_type(dtype):
    least, most = -2 ** 31, 2 ** 31 - 1
    x = tokens(17, 80, 1, 2, 128, 128, dtype)
    for off in ([0, 70, least, 80], [0, 70, most, 80], [least, 70, 70, 80], [most, least, 70, 80]):
        st = gb.new_status()
        S = torch.full((3, 2, 128, 128), 7.0, device="cuda")
        gb.gdn_prefill(*x, torch.tensor(off, dtype=torch.int32, device="cuda"), most, S_new=S, dev_status=st,
                       workspace=torch.empty(1 << 28, dtype=torch.uint8, device="cuda"))
        assert int(st.item()) == 32, off
        for i, (lo, hi) in enumerate(zip(off, off[1:])):
            if not 0 <= lo <= hi <= 80:
                assert bool((S[i] == 7.0).all()), (off, i)
                continue
            _, rS = OL.prefill(*[f64(t)[lo:hi] for t in x], [0, hi - lo])
            close(S[i:i + 1], rS, TOL_STATE[dtype])


def test_prefill_on_another_stream_and_in_a_graph():
    lengths = [300, 40]
    x = tokens(16, 340, 2, 4, 128, 128, BF)
    off = offsets(lengths)
    o, S = gb.gdn_prefill(*x, off, 300)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, S2 = torch.empty_like(o), torch.empty_like(S)
    torch.cuda.synchronize()
    gb.gdn_prefill(*x, off, 300, out=o2, S_new=S2, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2)
    o3, S3 = torch.zeros_like(o), torch.zeros_like(S)
    need = gb.gdn_prefill_workspace(2, 2, 4, 128, 128, 340, 300)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gb.gdn_prefill(*x, off, 300, out=o3, S_new=S3, workspace=ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o3) and torch.equal(S, S3)


def test_prefill_then_verify_then_commit_then_decode():
    """The operators around the tree: a prompt's state, a chain draft verified and committed on it, then
    single tokens, all equal to one long prompt."""
    T, hk, hv, d = 90, 2, 4, 128
    x = tokens(17, T, hk, hv, d, d, BF, slow=True)
    ro, rS = OL.prefill(*map(f64, x), [0, T])
    part = lambda lo, hi: [t[lo:hi] for t in x]  # noqa: E731
    o1, S = gb.gdn_prefill(*part(0, 70), offsets([70]), 70)
    q, k, v, g, beta = part(70, 86)
    parent = torch.arange(-1, 15, dtype=torch.int32, device="cuda")
    no = offsets([16])
    mask, depth = gb.gdn_tree_build_desc(parent, no, 16)
    o2 = gb.gdn_tree_verify(q, k, v, g, beta, S, no, parent, mask, depth, 16, max_depth=16)
    path = torch.arange(16, dtype=torch.int32, device="cuda")
    gb.gdn_tree_commit(k, v, g, beta, S, no, parent, no, path, 16, max_path=16, out=S)
    outs = [gb.gdn_decode(*part(t, t + 1), S) for t in range(86, T)]
    o = torch.cat([o1, o2] + outs)
    close(o, ro, TOL[BF])
    close(S, rS, TOL_STATE[BF])


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF, BF), (BF, F32)])
@pytest.mark.parametrize("batch,hk,hv,dk,dv", [(1, 1, 1, 16, 16), (1, 16, 32, 128, 128), (5, 2, 4, 64, 128), (3, 1, 3, 32, 64),
                                               (33, 2, 2, 128, 16), (4, 1, 2, 16, 128), (70, 2, 8, 128, 128)])
def test_decode(batch, hk, hv, dk, dv, dtype, out_dtype):
    x = tokens(batch, batch, hk, hv, dk, dv, dtype)
    S = pool(6, batch + 3, hv, dk, dv)
    before = f64(S)
    slots = torch.randperm(batch + 3, generator=torch.Generator().manual_seed(1))[:batch].to(torch.int32).cuda()
    slots[batch // 2] = -1 if batch > 1 else slots[0]
    st = gb.new_status()
    o = gb.gdn_decode(*x, S, slots=slots, scale=0.5, out_dtype=out_dtype, dev_status=st)
    gb.check_status(st)
    ro, rS = OL.decode(*map(f64, x), before, slots.cpu().numpy(), 0.5)
    close(o, ro, 2.0 ** -8 if out_dtype == BF else TOL[F32])
    close(S, rS, TOL_STATE[F32])
    unused = sorted(set(range(batch + 3)) - set(slots.tolist()))
    assert np.array_equal(f64(S)[unused], before[unused])
    if batch > 1:
        assert bool((o[batch // 2] == 0).all())


@pytest.mark.parametrize("pad", [0, 8, 3])
def test_decode_strided_rows_bad_slot_full_decay(pad):
    B, hk, hv, d = 4, 2, 4, 128
    q, k, v, g, beta = tokens(20, B, hk, hv, d, d, BF)
    g[2] = -float("inf")
    rows = torch.full((B, (2 * hk + hv) * d + pad), float("nan"), dtype=BF, device="cuda")
    qs = rows[:, :hk * d].view(B, hk, d)
    ks = rows[:, hk * d:2 * hk * d].view(B, hk, d)
    vs = rows[:, 2 * hk * d:(2 * hk + hv) * d].view(B, hv, d)
    qs.copy_(q), ks.copy_(k), vs.copy_(v)
    S = pool(7, 4, hv, d, d)
    before = f64(S)
    slots = torch.tensor([1, 9, 0, 3], dtype=torch.int32, device="cuda")
    st = gb.new_status()
    out = torch.full((B, hv, d), 7.0, dtype=BF, device="cuda")
    gb.gdn_decode(qs, ks, vs, g, beta, S, slots=slots, out=out, dev_status=st)
    assert int(st.item()) == 128
    assert bool((out[1] == 7.0).all())
    use = [0, 2, 3]
    ro, rS = OL.decode(*[f64(t)[use] for t in (q, k, v, g, beta)], before, [1, 0, 3])
    close(out[use], ro, 2.0 ** -8)
    close(S, rS, TOL_STATE[F32])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,hk,hv,dk,pad", [(1, 1, 1, 16, 0), (37, 2, 6, 32, 0), (5, 16, 32, 128, 0), (300, 1, 4, 64, 8),
                                            (9, 4, 4, 128, 3), (1000, 3, 3, 128, 0)])
def test_qk_gates(T, hk, hv, dk, pad, dtype):
    gen = torch.Generator().manual_seed(T)
    rows = (10.0 ** torch.randint(-3, 4, (T, 1), generator=gen) * torch.randn(T, 2 * hk * dk + pad, generator=gen)).to(dtype).cuda()
    q, k = rows[:, :hk * dk].view(T, hk, dk), rows[:, hk * dk:2 * hk * dk].view(T, hk, dk)
    q[0, 0] = 0.0
    ab = (8.0 * torch.randn(T, 2 * hv, generator=gen)).to(dtype).cuda()
    ab[0, 0], ab[-1, -1], ab[T // 2, hv] = 1000.0, -1000.0, 1000.0
    a, b = ab[:, :hv], ab[:, hv:]
    A_log, dt_bias = torch.randn(hv, generator=gen).cuda(), torch.randn(hv, generator=gen).cuda()
    got = gb.gdn_qk_gates(q, k, a, b, A_log, dt_bias, eps=1e-6)
    ref = OL.qk_gates(*map(f64, (q, k, a, b, A_log, dt_bias)), 1e-6)
    for x, r in zip(got[:2], ref[:2]):
        assert np.max(np.abs(f64(x) - r) - (2.0 ** -8 if dtype == BF else 2.0 ** -21) * np.abs(r)) <= 1e-12
    for x, r in zip(got[2:], ref[2:]):  # a few fp32 roundings and the functions' own few units
        assert np.max(np.abs(f64(x) - r) - 2.0 ** -19 * np.abs(r)) <= 1e-35


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("dtype,wtype", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,hv,dv,pad", [(1, 1, 16, 0), (7, 32, 128, 0), (129, 3, 64, 8), (50, 2, 32, 3), (600, 5, 128, 0)])
def test_norm_gate(T, hv, dv, pad, dtype, wtype, act):
    gen = torch.Generator().manual_seed(T)
    rows = torch.randn(T, 2 * hv * dv + pad, generator=gen).to(dtype).cuda()
    o, z = rows[:, :hv * dv].view(T, hv, dv), rows[:, hv * dv:2 * hv * dv].view(T, hv, dv)
    o[0, 0] = 0.0
    z[0, 0, 0], z[0, 0, 1] = 90.0, -200.0
    w = torch.randn(dv, generator=gen).to(wtype).cuda()
    y = gb.gdn_norm_gate(o, z, w, eps=1e-6, act=act)
    r = OL.norm_gate(f64(o), f64(z), f64(w), 1e-6, act)
    assert np.max(np.abs(f64(y) - r) - (2.0 ** -8 if dtype == BF else 2.0 ** -19) * np.abs(r)) <= 1e-30


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("dtype,wtype", [(F32, F32), (BF, BF), (BF, F32)])
@pytest.mark.parametrize("T,D,pad", [(1, 1, 0), (3, 7, 0), (5, 257, 0), (2, 64, 8), (400, 768, 0), (4, 4096, 0), (700, 1024, 8),
                                     (3, 20000, 0), (2, 65536, 0), (350, 5120, 0), (6, 1024, 3)])
def test_residual_norm(T, D, pad, dtype, wtype, post):
    gen = torch.Generator().manual_seed(D)
    x = (3.0 * torch.randn(T, D + pad, generator=gen)).to(dtype).cuda()[:, :D]
    y = torch.randn(T, D + 2 * pad, generator=gen).to(dtype).cuda()[:, :D]
    y[0] = 0.0
    w, pw = torch.randn(D, generator=gen).to(wtype).cuda(), torch.randn(D, generator=gen).to(wtype).cuda()
    h, n = gb.gdn_residual_norm(x, y, w, scale=0.7, post_weight=pw if post else None, eps=1e-6)
    rh, rn = OL.residual_norm(f64(x), f64(y), f64(w), np.float64(np.float32(0.7)), f64(pw) if post else None, 1e-6)
    # h is a sum of two terms that may cancel, each good to a few 2^-24, and is then rounded to its type
    size = np.abs(f64(x)) + np.abs(rh - f64(x))
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -22
    assert np.max(np.abs(f64(h) - rh) - half * np.abs(rh) - 2.0 ** -20 * size) <= 1e-12
    scale_n = np.abs(rn) / np.maximum(np.abs(rh), 1e-30) * size
    assert np.max(np.abs(f64(n) - rn) - half * np.abs(rn) - 2.0 ** -19 * scale_n) <= 1e-12
    if pad == 0:
        x2, y2 = x.clone(), y.clone()
        gb.gdn_residual_norm(x2, y2, w, scale=0.7, post_weight=pw if post else None, eps=1e-6, h=x2, out=y2)
        assert torch.equal(x2, h) and torch.equal(y2, n)


def test_example_serves_a_layer():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "layer_serving.py")
    spec = importlib.util.spec_from_file_location("layer_serving", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    stream, states = example.run()
    # the rule's bf16 outputs differ by their rounding, then pass a bf16 product and sum; q, k, v are the same bits
    # up to the products' own rounding of another batch
    assert stream <= 2.0 ** -5 and states <= 2.0 ** -6


def test_prefill_many_more_prompts_than_sms():
    rng = np.random.default_rng(3)
    lengths = rng.integers(0, 150, 230).tolist()
    x = tokens(22, sum(lengths), 1, 2, 128, 128, BF)
    off = offsets(lengths)
    st = gb.new_status()
    o, S = gb.gdn_prefill(*x, off, 150, dev_status=st)
    gb.check_status(st)
    ro, rS = OL.prefill(*map(f64, x), off.cpu().numpy())
    close(o, ro, TOL[BF])
    close(S, rS, TOL_STATE[BF])


@pytest.mark.parametrize("lengths", [[1] * 90, [3, 20, 28, 1] * 25])
def test_prefill_short_prompts_fill_the_gpu(lengths):
    x = tokens(23, sum(lengths), 1, 2, 128, 128, BF)
    off = offsets(lengths)
    S0 = pool(9, len(lengths), 2, 128, 128)
    o, S = gb.gdn_prefill(*x, off, 28, S0=S0)
    ro, rS = OL.prefill(*map(f64, x), off.cpu().numpy(), S0=f64(S0))
    close(o, ro, TOL[BF])
    close(S, rS, TOL_STATE[BF])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_and_states_past_2_to_the_31(dtype):
    # rows so far apart, and a slot so far into the pool, that offsets pass 32 bits
    T, hv, d = 90, 2, 128
    q, k, v, g, beta = tokens(24, T, 1, hv, d, d, dtype, slow=True)
    stride = 1 << 25
    rows = torch.empty(T * stride, dtype=dtype, device="cuda").view(T, stride)
    qs, ks, vs = rows[:, :d].view(T, 1, d), rows[:, d:2 * d].view(T, 1, d), rows[:, 2 * d:(2 + hv) * d].view(T, hv, d)
    qs.copy_(q), ks.copy_(k), vs.copy_(v)
    n = 70000
    S = torch.empty(n, hv, d, d, device="cuda")
    S0 = pool(10, 1, hv, d, d)
    S[n - 1] = S0[0]
    slots = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    o, _ = gb.gdn_prefill(qs[:80], ks[:80], vs[:80], g[:80], beta[:80], offsets([80]), 80, S0=S, S_new=S, slots=slots)
    outs = [gb.gdn_decode(qs[t:t + 1], ks[t:t + 1], vs[t:t + 1], g[t:t + 1], beta[t:t + 1], S, slots=slots) for t in range(80, T)]
    ro, rS = OL.prefill(*map(f64, (q, k, v, g, beta)), [0, T], S0=f64(S0))
    close(torch.cat([o] + outs), ro, TOL[dtype])
    close(S[n - 1:], rS, TOL_STATE[dtype])
    y = gb.gdn_norm_gate(vs, vs, torch.ones(d, device="cuda"))
    assert torch.equal(y, gb.gdn_norm_gate(v, v, torch.ones(d, device="cuda")))
    rest = (v[:, :, 0].contiguous(), v[:, :, 1].contiguous(), torch.zeros(hv, device="cuda"), torch.zeros(hv, device="cuda"))
    for got, ref in zip(gb.gdn_qk_gates(qs, ks, *rest), gb.gdn_qk_gates(q, k, *rest)):
        assert torch.equal(got, ref)


def test_prefill_wait_probe_reports_and_still_computes():
    x = tokens(25, 100, 1, 2, 128, 128, BF)
    ref, rS = gb.gdn_prefill(*x, offsets([100]), 100)
    st = gb.new_status()
    gb.gdn_test_set_wait_probe(1000)
    try:
        o, S = gb.gdn_prefill(*x, offsets([100]), 100, dev_status=st)
        torch.cuda.synchronize()
    finally:
        gb.gdn_test_set_wait_probe(0)
    assert int(st.item()) == 16
    assert torch.equal(o, ref) and torch.equal(S, rS)


def test_same_inputs_same_bits():
    lengths = [700, 64, 300, 1]
    x = tokens(26, sum(lengths), 2, 4, 128, 128, BF)
    first = gb.gdn_prefill(*x, offsets(lengths), 700)
    for _ in range(3):
        again = gb.gdn_prefill(*x, offsets(lengths), 700)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_binding_refusals():
    x = tokens(1, 4, 1, 2, 16, 16, F32)
    off = offsets([4])
    with pytest.raises(TypeError):
        gb.gdn_prefill(x[0].cpu(), *x[1:], off, 4)
    with pytest.raises(TypeError):
        gb.gdn_prefill(x[0], x[1].to(BF), *x[2:], off, 4)
    with pytest.raises(ValueError):
        gb.gdn_prefill(x[0], x[1][:3], *x[2:], off, 4)
    with pytest.raises(ValueError):
        gb.gdn_prefill(*x, off, 4, slots=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        gb.gdn_decode(*x, torch.zeros(3, 2, 16, 16, device="cuda"))
    with pytest.raises(ValueError):
        gb.gdn_decode(*x, torch.zeros(4, 2, 16, 32, device="cuda")[..., ::2])
    with pytest.raises(ValueError):
        gb.gdn_norm_gate(x[2], x[2], torch.ones(16, device="cuda"), act="gelu")
    with pytest.raises(ValueError):
        gb.gdn_residual_norm(torch.ones(4, 8, device="cuda").t(), torch.ones(8, 4, device="cuda"), torch.ones(4, device="cuda"))
    with pytest.raises(gb.GdnError):
        gb.gdn_qk_gates(x[0][:, :, :8].contiguous(), x[1][:, :, :8].contiguous(), x[3], x[4], x[3][0], x[3][0])


@pytest.mark.parametrize("dtype,dv", [(F32, 128), (BF, 128), (BF, 64)])
@pytest.mark.parametrize("batch", [2, 40, 128, 200, 256, 257])
def test_prefill_takes_prompts_in_any_order(dtype, dv, batch):
    # more items than the GPU holds at once, lengths with ties, empty and refused prompts among them
    lengths = [(7 * b * b + 3) % 90 if b % 5 else 0 for b in range(batch)]
    hv = 16 if batch < 40 else 8
    T = sum(lengths)
    x = tokens(31, T, 2, hv, 128, dv, dtype)
    off = offsets(lengths)
    slots = torch.arange(batch, dtype=torch.int32).flip(0).cuda()
    slots[0] = batch
    st = gb.new_status()
    S = torch.zeros(batch, hv, dv, 128, device="cuda")
    o, _ = gb.gdn_prefill(*x, off, 90, slots=slots, S_new=S, dev_status=st)
    assert int(st.item()) == 128
    at = off.tolist()
    for b in {1, batch // 2, batch - 2, batch - 1} - {0}:
        ro, rS = OL.prefill(*[f64(t)[at[b]:at[b + 1]] for t in x], [0, lengths[b]])
        close(o[at[b]:at[b + 1]], ro, TOL[dtype])
        i = int(slots[b])
        close(S[i:i + 1], rS, TOL_STATE[dtype])
    alone, _ = gb.gdn_prefill(*[t[at[1]:] for t in x], torch.tensor([0, lengths[1]], dtype=torch.int32, device="cuda"), 90)
    if batch >= 40:  # neither cut into segments: the same bits
        assert torch.equal(alone[:lengths[1]], o[at[1]:at[2]])


@pytest.mark.parametrize("T", [3, 5000])
def test_calls_one_after_the_other_eager_and_in_a_graph(T):
    # each call reads what the one before wrote, in a stream that ends and begins with torch's own kernels
    hk, hv, d = 2, 4, 128
    x = torch.randn(T, (2 * hk + 2 * hv) * d + 2 * hv, generator=torch.Generator().manual_seed(41)).to(BF).cuda()
    cut = [0, hk * d, 2 * hk * d, (2 * hk + hv) * d, (2 * hk + 2 * hv) * d, (2 * hk + 2 * hv) * d + hv, x.shape[1]]
    A_log, dt_bias = torch.linspace(-1, 1, hv).cuda(), torch.linspace(-2, 0, hv).cuda()
    w, wr = torch.linspace(.5, 1.5, d).to(BF).cuda(), torch.linspace(.5, 1.5, hv * d).to(BF).cuda()
    S0 = pool(42, T, hv, d, d)
    slots = torch.arange(T, dtype=torch.int32, device="cuda").flip(0)

    def chain(S, wait):
        S.copy_(S0)
        y = x
        for _ in range(3):
            parts = [y[:, a:b] for a, b in zip(cut, cut[1:])]
            q, k = parts[0].view(T, hk, d), parts[1].view(T, hk, d)
            v, z = parts[2].view(T, hv, d), parts[3].view(T, hv, d)
            q, k, g, beta = gb.gdn_qk_gates(q, k, parts[4], parts[5], A_log, dt_bias)
            wait()
            o = gb.gdn_decode(q, k, v, g, beta, S, slots)
            wait()
            o = gb.gdn_norm_gate(o, z, w)
            wait()
            h, n = gb.gdn_residual_norm(o.view(T, hv * d), parts[2], wr)
            wait()
            y = torch.cat([n, h, n, y[:, cut[4]:]], dim=1)
        return y

    S1, S2, S3 = torch.empty_like(S0), torch.empty_like(S0), torch.empty_like(S0)
    ref = chain(S1, torch.cuda.synchronize)
    got = chain(S2, lambda: None)
    assert torch.equal(ref, got) and torch.equal(S1, S2)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        y = chain(S3, lambda: None)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ref, y) and torch.equal(S1, S3)
