"""The scan and its gradients against the recurrence token by token in 64 bits (tests/layer_reference.py, which also
derives the tolerances)."""
import pytest
import torch

import linear_attention_recurrent_decode_b200 as kda
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu
K = V = 128
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dstate")


def inputs(lens, H, decay="softplus", seed=0, gap=0, tail=0, dev="cuda"):
    """q, k, v, g, beta, cu_seqlens of sequences of these lengths, `gap` rows ahead of them and `tail` behind."""
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    T = gap + sum(lens) + tail
    unit = [x / x.norm(dim=-1, keepdim=True) for x in (randn(T, H, K), randn(T, H, K))]
    sp = -torch.nn.functional.softplus(randn(T, H, K))
    if decay == "softplus":
        g = sp
    elif decay == "mild":
        g = sp * 0.05
    elif decay == "none":
        g = torch.zeros(T, H, K, device=dev)
    elif decay == "strong":       # out of the factors' range in most sub-blocks
        g = sp * 30
    elif decay == "mixed":        # a few channels far out of range, some at once, some forgetting everything
        g = sp.clone()
        g[:, :, :8] = -25.0
        g[::7, :, 8:12] = -1e5
        g[::5, :, 12:14] = float("-inf")
    elif decay == "growing":
        g = 0.02 * randn(T, H, K)
    beta = torch.sigmoid(randn(T, H))
    cu = [gap]
    for n in lens:
        cu.append(cu[-1] + n)
    return unit[0].bfloat16(), unit[1].bfloat16(), randn(T, H, V).bfloat16(), g, beta, torch.tensor(cu, dtype=torch.int32, device=dev)


def states(N, H, seed, scale=0.3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(N, H, K, V, generator=gen, device="cuda") * scale


def double(*xs):
    return [x.double() for x in xs]


def check_scan(out, final, q, k, v, g, beta, state, cu, scale):
    ro, rs = ref.scan(*double(q, k, v, g, beta), state.double(), cu, scale)
    floor = ref.FLOOR * max(float(x.abs().max()) for x in (v, state) if x.numel())
    for n in range(len(cu) - 1):  # a sequence's results are held to its own magnitude
        a, b = int(cu[n]), int(cu[n + 1])
        if b > a:
            ref.check(out[a:b], ro[a:b], ref.SCAN_REL, f"out of sequence {n}", ref.BF16_HALF_STEP, floor * scale)
        ref.check(final[n], rs[n], ref.SCAN_REL, f"state of sequence {n}", floor=floor)


LENGTHS = [
    ([1], 1), ([2], 3), ([16], 2), ([17, 15, 1], 2), ([63, 64, 65], 2), ([128], 1), ([129, 0, 31], 2), ([0, 5, 0, 0, 70, 0], 1),
    ([100, 1, 219], 4), ([7] * 40, 3), ([300, 200], 16), ([90] * 8, 20),
]
# walked in segments of 8 chunks: one to five of them, the last from one token to full
LONG = [([64 * 24], 2), ([1600], 1), ([64 * 16 + 1, 0, 500, 64 * 8], 2), ([2100, 1, 70], 1)]
LONG += [([64 * 13, 64 * 13 + 1, 3, 64 * 9 + 5, 64 * 14], 2)]  # cut as the longest has 14 chunks


@pytest.mark.parametrize("lens,H", LENGTHS + LONG)
@pytest.mark.parametrize("with_state", [False, True])
def test_scan_lengths(lens, H, with_state, cuda_device):
    q, k, v, g, beta, cu = inputs(lens, H, "mild" if (lens, H) in LONG else "softplus", seed=len(lens) + H)
    state = states(len(lens), H, 5) if with_state else None
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu)
    check_scan(out, final, q, k, v, g, beta, state if with_state else torch.zeros_like(final), cu.tolist(), K ** -0.5)


@pytest.mark.parametrize("decay", ["softplus", "mild", "none", "strong", "mixed", "growing"])
@pytest.mark.parametrize("edge", ["", "beta0", "beta1", "zero_v", "zero_k"])
def test_scan_decays_and_edges(decay, edge, cuda_device):
    q, k, v, g, beta, cu = inputs([130, 37], 2, decay, seed=11)
    if edge == "beta0":
        beta.zero_()
    elif edge == "beta1":
        beta.fill_(1.0)
    elif edge == "zero_v":
        v.zero_()
    elif edge == "zero_k":
        k.zero_()
    state = states(2, 2, 6)
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu, scale=0.7)
    check_scan(out, final, q, k, v, g, beta, state, cu.tolist(), 0.7)


@pytest.mark.parametrize("magnitude", [2.0 ** -30, 2.0 ** -12, 1.0, 2.0 ** 12, 2.0 ** 30])
def test_scan_magnitudes(magnitude, cuda_device):
    """Values and states of any size: the operand pairs are scaled to their tile."""
    q, k, v, g, beta, cu = inputs([150], 2, seed=12)
    v, state = v * magnitude, states(1, 2, 6) * magnitude
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu)
    check_scan(out, final, q, k, v, g, beta, state, cu.tolist(), K ** -0.5)


def test_scan_dense_form_equals_packed(cuda_device):
    N, T, H = 3, 150, 2
    q, k, v, g, beta, cu = inputs([T] * N, H, seed=3)
    state = states(N, H, 4)
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu)
    dense = [x.view(N, T, *x.shape[1:]) for x in (q, k, v, g, beta)]
    out2, final2 = kda.kda_scan(*dense, state)
    assert torch.equal(out2.view_as(out), out) and torch.equal(final2, final)
    one = [x[:1, :1] for x in dense]  # a single token
    out3, final3 = kda.kda_scan(*one, state[:1])
    check_scan(out3[0], final3, *(x[0] for x in one), state[:1], [0, 1], K ** -0.5)
    empty = kda.kda_scan(*(x[:, :0] for x in dense), state)
    assert empty[0].shape == (N, 0, H, V) and torch.equal(empty[1], state)
    nothing = kda.kda_scan(*(x[:0] for x in dense))
    assert nothing[0].shape == (0, T, H, V) and nothing[1].shape == (0, H, K, V)


def test_scan_strided_rows_gaps_and_untouched_memory(cuda_device):
    """q, k, v as slices of one buffer, g, beta and out with strides of their own; rows outside every sequence hold NaN,
    are not read, and keep what the output had there."""
    H, lens, gap, tail = 3, [70, 33], 5, 9
    q, k, v, g, beta, cu = inputs(lens, H, seed=21, gap=gap, tail=tail)
    T = q.shape[0]
    inside = torch.zeros(T, dtype=torch.bool, device=cuda_device)
    inside[gap:T - tail] = True
    want, wfinal = kda.kda_scan(q, k, v, g, beta, cu_seqlens=cu)
    packed = torch.full((T, 3 * H * K + 8), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    qs, ks, vs = (packed[:, i * H * K:(i + 1) * H * K].unflatten(-1, (H, K)) for i in range(3))
    gs = torch.full((T, H * K + 3), float("nan"), device=cuda_device)[:, :H * K].unflatten(-1, (H, K))
    bs = torch.full((T, 5 * H), float("nan"), device=cuda_device)[:, H:2 * H]
    outs = torch.full((T, 2 * H * V), 7.0, dtype=torch.bfloat16, device=cuda_device)
    for dst, src in ((qs, q), (ks, k), (vs, v), (gs, g), (bs, beta)):
        dst[inside] = src[inside]
    out = outs[:, H * V:].unflatten(-1, (H, V))
    got, final = kda.kda_scan(qs, ks, vs, gs, bs, cu_seqlens=cu, out=out)
    assert got is out and torch.equal(out[inside], want[inside]) and torch.equal(final, wfinal)
    assert bool((out[~inside] == 7).all()) and bool((outs[:, :H * V] == 7).all())
    # the gradients too
    d_out = torch.randn(T, H, V, device=cuda_device).bfloat16()
    want = kda.kda_scan_backward(d_out, q, k, v, g, beta, cu_seqlens=cu)
    d_out[~inside] = float("nan")
    buf = torch.full((T, 3 * H * K + 8), 7.0, dtype=torch.bfloat16, device=cuda_device)
    dq, dk, dv = (buf[:, i * H * K:(i + 1) * H * K].unflatten(-1, (H, K)) for i in range(3))
    dg = torch.full((T, H * K + 3), 7.0, device=cuda_device)[:, :H * K].unflatten(-1, (H, K))
    dbeta = torch.full((T, 2 * H), 7.0, device=cuda_device)[:, :H]
    got = kda.kda_scan_backward(d_out, qs, ks, vs, gs, bs, cu_seqlens=cu, dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta)
    for name, a, b in zip(GRADS[:5], got, want):
        assert torch.equal(a[inside], b[inside]), name
        assert bool((a[~inside] == 7).all()), name
    assert torch.equal(got[5], want[5]) and bool((buf[:, 3 * H * K:] == 7).all())


def test_scan_slots(cuda_device):
    """States in a pool: updated in place or from one pool to another, inactive sequences, other blocks untouched."""
    H, lens = 2, [65, 20, 0, 30, 64]
    q, k, v, g, beta, cu = inputs(lens, H, seed=31)
    pool = states(7, H, 8)
    slots = torch.tensor([4, -1, 0, 7, 2], dtype=torch.int32, device=cuda_device)  # 1: padding, 3: beyond the pool
    before, c = pool.clone(), cu.tolist()
    out, final = kda.kda_scan(q, k, v, g, beta, pool, cu_seqlens=cu, slot_idx=slots)
    assert final is pool
    for n, s in ((0, 4), (2, 0), (4, 2)):
        a, b = c[n], c[n + 1]
        check_scan(out[a:b], pool[s:s + 1], q[a:b], k[a:b], v[a:b], g[a:b], beta[a:b], before[s:s + 1], [0, b - a], K ** -0.5)
    for n in (1, 3):
        assert bool((out[c[n]:c[n + 1]] == 0).all())
    for s in (1, 3, 5, 6):
        assert torch.equal(pool[s], before[s])
    other = torch.full_like(pool, 3.0)
    out2, final2 = kda.kda_scan(q, k, v, g, beta, before, cu_seqlens=cu, slot_idx=slots, final_state=other)
    assert final2 is other and torch.equal(out2, out)
    for s in range(7):
        assert torch.equal(other[s], pool[s]) if s in (4, 0, 2) else bool((other[s] == 3).all())


def test_scan_slots_of_long_sequences(cuda_device):
    """In place through segments, with an inactive sequence among them; and the dense form's segments."""
    H, lens = 2, [1300, 900, 600]
    q, k, v, g, beta, cu = inputs(lens, H, "mild", seed=32)
    pool, c = states(4, H, 8), cu.tolist()
    slots = torch.tensor([3, -1, 0], dtype=torch.int32, device=cuda_device)
    before = pool.clone()
    out, _ = kda.kda_scan(q, k, v, g, beta, pool, cu_seqlens=cu, slot_idx=slots)
    for n, s in ((0, 3), (2, 0)):
        a, b = c[n], c[n + 1]
        check_scan(out[a:b], pool[s:s + 1], q[a:b], k[a:b], v[a:b], g[a:b], beta[a:b], before[s:s + 1], [0, b - a], K ** -0.5)
    assert bool((out[c[1]:c[2]] == 0).all()) and torch.equal(pool[1:3], before[1:3])
    T = 1700  # two sequences of 27 chunks
    q, k, v, g, beta, cu = inputs([T] * 2, 1, "mild", seed=33)
    state = states(2, 1, 4)
    out, final = kda.kda_scan(*(x.view(2, T, *x.shape[1:]) for x in (q, k, v, g, beta)), state)
    check_scan(out.view(2 * T, 1, V), final, q, k, v, g, beta, state, cu.tolist(), K ** -0.5)


def test_scan_long_sequences_in_place(cuda_device):
    """The last segment of a sequence, here of one token, stores the final state while the first may not have started: the
    walk of the results takes the initial state from a copy in the workspace, made by the kernel before."""
    H, T = 3, 64 * 24 + 1
    q, k, v, g, beta, cu = inputs([T], H, "mild", seed=34)
    start, pool = states(1, H, 8), states(3, H, 9)
    want, wfinal = kda.kda_scan(q, k, v, g, beta, start, cu_seqlens=cu)
    check_scan(want, wfinal, q, k, v, g, beta, start, cu.tolist(), K ** -0.5)
    pool[2] = start[0]
    ws = torch.zeros(kda.scan_workspace_bytes(T, 1, H), dtype=torch.uint8, device=cuda_device)
    slots = torch.tensor([2], dtype=torch.int32, device=cuda_device)
    out, _ = kda.kda_scan(q, k, v, g, beta, pool, cu_seqlens=cu, slot_idx=slots, workspace=ws)
    assert torch.equal(out, want) and torch.equal(pool[2], wfinal[0])
    blocks = ws[ws.numel() % (K * V * 4):].view(torch.float32).view(-1, K, V)  # the segments' states lie at the end
    for h in range(H):
        assert bool((blocks == start[0, h]).all(-1).all(-1).any()), f"no copy of head {h}'s start"
    state = start.clone()
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu, final_state=state)
    assert final is state and torch.equal(out, want) and torch.equal(state, wfinal)


def test_scan_in_place_captured_and_at_once(cuda_device):
    """Pools that long sequences update in place: one by a graph replayed on one stream, one eagerly on another, three times
    each, as one after the other."""
    H, T = 2, 64 * 30 + 5
    x, y = inputs([T], H, "mild", seed=36), inputs([T, 100], H, "mild", seed=37)
    slots = [torch.tensor(s, dtype=torch.int32, device=cuda_device) for s in ([1], [2, 0])]

    def step(z, pool, i):
        return kda.kda_scan(*z[:5], pool, cu_seqlens=z[5], slot_idx=slots[i])[0]

    want = [states(3, H, 8), states(3, H, 9)]
    pools = [p.clone() for p in want]
    outs = [[step(z, p, i) for _ in range(3)][-1] for i, (z, p) in enumerate(zip((x, y), want))]
    graph, one, two = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        first = step(x, pools[0], 0)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(one):
            graph.replay()
        with torch.cuda.stream(two):
            second = step(y, pools[1], 1)
    torch.cuda.synchronize()
    assert torch.equal(first, outs[0]) and torch.equal(second, outs[1])
    assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1])


def test_scan_sequences_that_are_not_cut(cuda_device):
    """Sequences of 13 chunks where segments have 8 would be walked for longer in segments: nothing is written where the
    segments' states would be."""
    H, lens = 2, [64 * 13] * 2
    q, k, v, g, beta, cu = inputs(lens, H, "mild", seed=35)
    ws = torch.zeros(kda.scan_workspace_bytes(sum(lens), 2, H), dtype=torch.uint8, device=cuda_device)
    out, final = kda.kda_scan(q, k, v, g, beta, cu_seqlens=cu, workspace=ws)
    check_scan(out, final, q, k, v, g, beta, torch.zeros_like(final), cu.tolist(), K ** -0.5)
    slots = 26 // 8 + 2  # of segments
    assert not bool(ws[-2 * slots * H * K * V * 4:].any())


def test_scan_many_sequences(cuda_device):
    """More sequences than one, and than two, steps of the search for a chunk's sequence, of 0 to 3 tokens but for a long
    one, some without any at both ends."""
    lens = [0, 0] + [(n * 7) % 4 for n in range(1500)] + [70] + [(n * 5) % 4 for n in range(700)] + [0]
    q, k, v, g, beta, cu = inputs(lens, 1, seed=50, tail=3)
    state = states(len(lens), 1, 8)
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu)
    d_out, d_final = torch.ones_like(v), states(len(lens), 1, 9)
    got = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu)
    c = cu.tolist()
    for n in (0, 1, 2, 3, 4, 31, 32, 33, 1023, 1024, 1025, 1501, 1502, 1503, 2000, len(lens) - 2, len(lens) - 1):
        rows = slice(c[n], c[n + 1])
        x = [t[rows].contiguous() for t in (q, k, v, g, beta)]
        one = torch.tensor([0, lens[n]], dtype=torch.int32, device="cuda")
        o, f = kda.kda_scan(*x, state[n:n + 1], cu_seqlens=one)
        d = kda.kda_scan_backward(d_out[rows].contiguous(), *x, state[n:n + 1], d_final_state=d_final[n:n + 1], cu_seqlens=one)
        assert torch.equal(out[rows], o) and torch.equal(final[n], f[0]), n
        assert all(torch.equal(a[rows], b) for a, b in zip(got[:5], d)) and torch.equal(got[5][n], d[5][0]), n
    for a, b in zip(c, c[1:]):
        assert bool(torch.isfinite(out[a:b]).all()) and bool(torch.isfinite(got[3][a:b]).all())


def test_scan_no_tokens_is_ordered_behind_the_stream(cuda_device):
    """Dense sequences of no token: the states of the named slots pass through, named by work still in flight."""
    pool, final = states(6, 2, 12), torch.zeros(6, 2, K, V, device="cuda")
    slots = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    big = torch.randn(4096, 4096, device="cuda")
    empty = [torch.empty(3, 0, 2, w, dtype=t, device="cuda") for w, t in ((K, torch.bfloat16),) * 3 + ((K, torch.float32),)]
    beta = torch.empty(3, 0, 2, device="cuda")
    big @ big
    slots.copy_(torch.tensor([4, 0, 2], device="cuda"))
    kda.kda_scan(*empty, beta, pool, slot_idx=slots, final_state=final)
    want = torch.zeros_like(final)
    want[[4, 0, 2]] = pool[[4, 0, 2]]
    assert torch.equal(final, want)


def test_scan_bad_offsets_stay_in_bounds(cuda_device):
    """Offsets that decrease or leave the rows are clamped: an error in them cannot reach other memory."""
    q, k, v, g, beta, _ = inputs([100], 2, seed=41)
    cu = torch.tensor([-5, 60, 40, 1000, 2 ** 31 - 1], dtype=torch.int32, device=cuda_device)
    guard = torch.full((300, 2, V), 5.0, dtype=torch.bfloat16, device=cuda_device)
    out = guard[100:200]
    kda.kda_scan(q, k, v, g, beta, cu_seqlens=cu, out=out)
    torch.cuda.synchronize()
    assert bool((guard[:100] == 5).all()) and bool((guard[200:] == 5).all())
    # with segments
    q, k, v, g, beta, _ = inputs([2000], 1, seed=42)
    cu = torch.tensor([1990, 0, 2000, 3, 2 ** 31 - 1], dtype=torch.int32, device=cuda_device)
    guard = torch.full((2200, 1, V), 5.0, dtype=torch.bfloat16, device=cuda_device)
    kda.kda_scan(q, k, v, g, beta, cu_seqlens=cu, out=guard[100:2100])
    torch.cuda.synchronize()
    assert bool((guard[:100] == 5).all()) and bool((guard[2100:] == 5).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scan_nan_stays_in_its_sequence_and_head(bad, cuda_device):
    q, k, v, g, beta, cu = inputs([70, 130, 40], 2, seed=51)
    d_out = torch.randn(240, 2, V, device=cuda_device).bfloat16()
    want, wfinal = kda.kda_scan(q, k, v, g, beta, cu_seqlens=cu)
    wgrad = kda.kda_scan_backward(d_out, q, k, v, g, beta, cu_seqlens=cu)
    v[70 + 100, 1, 3] = bad  # sequence 1, its second chunk, head 1
    k[70 + 101, 1, 5] = bad
    out, final = kda.kda_scan(q, k, v, g, beta, cu_seqlens=cu)
    grads = kda.kda_scan_backward(d_out, q, k, v, g, beta, cu_seqlens=cu)
    same = torch.ones(240, 2, dtype=torch.bool, device=cuda_device)
    same[70:200, 1] = False
    assert torch.equal(out[same], want[same]) and torch.equal(out[70:134, 1], want[70:134, 1])
    ok = torch.tensor([[1, 1], [1, 0], [1, 1]], dtype=torch.bool, device=cuda_device)
    assert torch.equal(final[ok], wfinal[ok])
    for name, a, b in zip(GRADS, grads, wgrad):
        m = ok if name == "dstate" else same
        assert torch.equal(a[m], b[m]), name


def check_gradients(got, want, cu, q, k, d_out, d_final):
    """Each sequence's gradients to their own magnitude.  Values and states are of the order of 1 here, so the largest input
    of the gradients' recurrence is that of d_out and d_final."""
    floor = ref.FLOOR * max(float(d_out.abs().max()), 0.0 if d_final is None else float(d_final.abs().max()))
    for name, a, b in zip(GRADS, got, want):
        rel = ref.DG_REL if name == "dg" else ref.SCAN_REL
        step = ref.BF16_HALF_STEP if name in ("dq", "dk", "dv") else 0.0
        for n in range(len(cu) - 1):
            lo, hi = (n, n + 1) if name == "dstate" else (int(cu[n]), int(cu[n + 1]))
            if hi > lo:
                terms = 0.0
                if name == "dg":
                    terms = rel * float((q[lo:hi].double() * want[0][lo:hi]).abs().max() + (k[lo:hi].double() * want[1][lo:hi]).abs().max())
                ref.check(a[lo:hi], b[lo:hi], rel, f"{name} of sequence {n}", step, floor + terms)


@pytest.mark.parametrize("lens,H", [x for x in LENGTHS if sum(x[0]) * x[1] < 4000] + LONG)
@pytest.mark.parametrize("with_state", [False, True])
def test_scan_gradients_lengths(lens, H, with_state, cuda_device):
    q, k, v, g, beta, cu = inputs(lens, H, "mild" if (lens, H) in LONG else "softplus", seed=61 + H)
    N, c = len(lens), cu.tolist()
    d_out = torch.randn(sum(lens), H, V, device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(1)).bfloat16()
    state = states(N, H, 5) if with_state else None
    d_final = states(N, H, 6) if with_state else None
    zero = torch.zeros(N, H, K, V, device=cuda_device)
    want = ref.scan_gradients(q, k, v, g, beta, zero if state is None else state, c, K ** -0.5, d_out, zero if d_final is None else d_final)
    ws = torch.empty(kda.scan_workspace_bytes(sum(lens), N, H, training=True), dtype=torch.uint8, device=cuda_device)
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu, workspace=ws, save=True)
    got = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu, workspace=ws, saved=True)
    again = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu)
    for name, a, b in zip(GRADS, got, again):
        assert torch.equal(a, b), f"{name}: computed from the saved pass and anew"
    check_gradients(got, want[2:], c, q, k, d_out, d_final)


@pytest.mark.parametrize("decay", ["softplus", "mild", "none", "strong", "mixed", "growing"])
@pytest.mark.parametrize("edge", ["", "beta0", "beta1", "zero_d_out", "zero_k"])
def test_scan_gradients_decays_and_edges(decay, edge, cuda_device):
    q, k, v, g, beta, cu = inputs([130, 37], 2, decay, seed=71)
    d_out = torch.randn(167, 2, V, device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(2)).bfloat16()
    if edge == "beta0":
        beta.zero_()
    elif edge == "beta1":
        beta.fill_(1.0)
    elif edge == "zero_d_out":
        d_out.zero_()
    elif edge == "zero_k":
        k.zero_()
    state, d_final, c = states(2, 2, 6), states(2, 2, 7), cu.tolist()
    want = ref.scan_gradients(q, k, v, g, beta, state, c, 0.7, d_out, d_final)
    got = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu, scale=0.7)
    check_gradients(got, want[2:], c, q, k, d_out, d_final)


@pytest.mark.parametrize("decay", ["softplus", "mild"])
def test_scan_decay_gradients_normwise(decay, cuda_device):
    """dg is what crosses each token: as a sum of rows minus columns over the rest of the chunk, strong decays would leave
    it as a small difference of large sums."""
    q, k, v, g, beta, cu = inputs([300, 64, 20], 2, decay, seed=75)
    d_out = torch.randn(384, 2, V, device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(3)).bfloat16()
    state, d_final, c = states(3, 2, 6, 0.02), states(3, 2, 7, 0.02), cu.tolist()
    want = ref.scan_gradients(q, k, v, g, beta, state, c, K ** -0.5, d_out, d_final)[5]
    got = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu)[3]
    for a, b in zip(c, c[1:]):
        assert float((got[a:b].double() - want[a:b]).norm() / want[a:b].norm()) <= ref.DG_NORM


@pytest.mark.parametrize("magnitude", [2.0 ** -80, 2.0 ** -60, 2.0 ** -45, 2.0 ** 45, 2.0 ** 70, 2.0 ** 95])
def test_scan_far_magnitudes(magnitude, cuda_device):
    """Near both ends of the documented range, 2^-80 to 2^100; the largest of these values and states is near 2^3."""
    q, k, v, g, beta, cu = inputs([150], 2, "mild", seed=13)
    v, state = v * magnitude, states(1, 2, 6) * magnitude
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu)
    check_scan(out, final, q, k, v, g, beta, state, cu.tolist(), K ** -0.5)


@pytest.mark.parametrize("mv,md", [(1.0, 2.0 ** -80), (1.0, 2.0 ** 90), (2.0 ** -70, 2.0 ** 90), (2.0 ** 90, 2.0 ** -70), (2.0 ** -45, 2.0 ** -30)])
def test_scan_gradients_far_magnitudes(mv, md, cuda_device):
    """A power of two on the values or on the gradients changes nothing but the results' exponents, other than where fp32
    ends at 2^-149, which is less than 2^-36 of these results' largest."""
    q, k, v, g, beta, cu = inputs([150, 30], 2, "mild", seed=14)
    state, d_final = states(2, 2, 6), states(2, 2, 7)
    d_out = torch.randn(180, 2, V, device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(4)).bfloat16()
    want = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu)
    check_gradients(want, ref.scan_gradients(q, k, v, g, beta, state, cu.tolist(), K ** -0.5, d_out, d_final)[2:], cu.tolist(), q, k,
                    d_out, d_final)
    got = kda.kda_scan_backward(d_out * md, q, k, v * mv, g, beta, state * mv, d_final_state=d_final * md, cu_seqlens=cu)
    for name, a, b in zip(GRADS, got, want):
        m = md if name in ("dv", "dstate") else mv * md
        ref.check(a, b.double() * m, ref.FLOOR, name, ref.BF16_HALF_STEP if name in ("dq", "dk", "dv") else 0.0)


def test_scan_columns_of_different_magnitude(cuda_device):
    """Value columns from 1 down to 2^-16 under one scale (32 columns share one): a pair's 2^-39 of the largest is still
    within 2^-23 of the smallest column's own, so each column is held to its own magnitude; and its gradients likewise."""
    q, k, v, g, beta, cu = inputs([150, 30], 2, "mild", seed=15)
    size = torch.exp2(-16.0 * (torch.arange(V, device=cuda_device) % 32) / 31).bfloat16()
    v, state, d_final = v * size, states(2, 2, 6) * size, states(2, 2, 7) * size
    d_out = torch.randn(180, 2, V, device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(5)).bfloat16() * size
    c = cu.tolist()
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu)
    grads = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu)
    want = ref.scan_gradients(q, k, v, g, beta, state, c, K ** -0.5, d_out, d_final)
    for i in range(V):
        ref.check(out[..., i], want[0][..., i], ref.SCAN_REL, f"out, column {i}", ref.BF16_HALF_STEP)
        ref.check(final[..., i], want[1][..., i], ref.SCAN_REL, f"state, column {i}")
        ref.check(grads[2][..., i], want[4][..., i], ref.SCAN_REL, f"dv, column {i}", ref.BF16_HALF_STEP)
        ref.check(grads[5][..., i], want[7][..., i], ref.SCAN_REL, f"dstate, column {i}")
    check_gradients(grads, want[2:], c, q, k, d_out, d_final)


def test_scan_growth_over_a_chunk(cuda_device):
    """Decays that grow, by the documented 2^16 over a chunk of 64 tokens, then fall: a token's operands are up to 2^16 below
    the chunk's largest, whose 2^-39 is 2^-23 of theirs, so each token's outputs are held to their own magnitude."""
    q, k, v, g, beta, cu = inputs([128], 2, seed=16)
    g[:64], g[64:] = 0.173, -0.173  # 64 of them: 2^15.97
    state = states(1, 2, 6)
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu)
    d_out, d_final = torch.ones_like(v), states(1, 2, 7)
    want = ref.scan_gradients(q, k, v, g, beta, state, cu.tolist(), K ** -0.5, d_out, d_final)
    for t in range(128):
        for h in range(2):
            ref.check(out[t, h], want[0][t, h], ref.SCAN_REL, f"out of token {t}, head {h}", ref.BF16_HALF_STEP)
    ref.check(final, want[1], ref.SCAN_REL, "state")
    got = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu)
    check_gradients(got, want[2:], cu.tolist(), q, k, d_out, d_final)


def test_scan_gradients_against_differences(cuda_device):
    """The directional derivative of the 64-bit loss, by central differences, against the kernel's gradients."""
    q, k, v, g, beta, cu = inputs([90, 40], 2, seed=81)
    c, state, d_final = cu.tolist(), states(2, 2, 8), states(2, 2, 9)
    d_out = torch.randn(130, 2, V, device=cuda_device).bfloat16()
    grads = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu)
    x = double(q, k, v, g, beta, state)
    dirs = [torch.randn_like(t) for t in x]

    def loss(eps):
        out, final = ref.scan(*(a + eps * d for a, d in zip(x, dirs)), c, K ** -0.5)
        return float((out * d_out.double()).sum() + (final * d_final.double()).sum())

    eps = 1e-6  # the third derivative's eps^2 and the loss's 2^-53 / eps are both far below the bound
    numeric = (loss(eps) - loss(-eps)) / (2 * eps)
    analytic = sum(float((gr.double() * d).sum()) for gr, d in zip(grads, dirs))
    # the bf16 gradients' rounding: half a step of every term
    bound = sum(float((gr.double() * d).abs().sum()) for gr, d in zip(grads[:3], dirs)) * ref.BF16_HALF_STEP
    assert abs(numeric - analytic) <= bound + 1e-3


@pytest.mark.parametrize("which", range(6), ids=GRADS)
def test_scan_each_gradient_against_differences(which, cuda_device):
    """The derivative of the 64-bit loss along one input at a time, by central differences, so that no gradient hides behind
    a larger one's rounding."""
    q, k, v, g, beta, cu = inputs([90, 40], 2, seed=82)
    gen = torch.Generator(device=cuda_device).manual_seed(83 + which)
    c, state, d_final = cu.tolist(), states(2, 2, 8), states(2, 2, 9)
    d_out = torch.randn(130, 2, V, device=cuda_device, generator=gen).bfloat16()
    grad = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu)[which].double()
    x = double(q, k, v, g, beta, state)
    way = torch.randn(x[which].shape, device=cuda_device, generator=gen, dtype=torch.float64)
    # along the gradient's signs: the terms add up instead of cancelling
    way = way.abs() * torch.where(grad < 0, -1.0, 1.0)

    def loss(eps):
        y = list(x)
        y[which] = y[which] + eps * way
        out, final = ref.scan(*y, c, K ** -0.5)
        return float((out * d_out.double()).sum() + (final * d_final.double()).sum())

    eps = 1e-6
    numeric, terms = (loss(eps) - loss(-eps)) / (2 * eps), float((grad * way).sum())
    # Per element: half a step where the gradient is bf16, and the tolerance of its largest.  The differences' own error is
    # the loss's 2^-53 / eps, with a loss below 2^12 5e-7 of 1, and eps^2 of the third derivative.
    rel = ref.DG_REL if which == 3 else ref.SCAN_REL
    bound = (ref.BF16_HALF_STEP * terms if which < 3 else 0.0) + 2 * rel * float(grad.abs().max() * way.abs().sum()) + 1e-4
    assert abs(numeric - terms) <= bound
    assert bound <= 0.05 * terms, "the bound would not see a gradient of zero"


def test_scan_dense_gradients_equal_packed(cuda_device):
    N, T, H = 2, 100, 2
    q, k, v, g, beta, cu = inputs([T] * N, H, seed=91)
    d_out, state, d_final = torch.randn(N * T, H, V, device=cuda_device).bfloat16(), states(N, H, 1), states(N, H, 2)
    a = kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu)
    b = kda.kda_scan_backward(*(x.view(N, T, *x.shape[1:]) for x in (d_out, q, k, v, g, beta)), state, d_final_state=d_final)
    for name, x, y in zip(GRADS, a, b):
        assert torch.equal(x, y.view_as(x)), name
    empty = kda.kda_scan_backward(*(x.view(N, T, *x.shape[1:])[:, :0] for x in (d_out, q, k, v, g, beta)), state, d_final_state=d_final)
    assert torch.equal(empty[5], d_final)


def test_scan_streams_graphs_and_repeats(cuda_device):
    """The same bits on another stream, twice at once with workspaces of their own, and replayed from two graphs that
    share a workspace in order; a graph reads its inputs anew."""
    H, lens = 4, [200, 77]
    q, k, v, g, beta, cu = inputs(lens, H, seed=101)
    d_out, state, d_final = torch.randn(277, H, V, device=cuda_device).bfloat16(), states(2, H, 1), states(2, H, 2)

    def step(**kw):
        ws = torch.empty(kda.scan_workspace_bytes(277, 2, H, training=True), dtype=torch.uint8, device=cuda_device)
        out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu, workspace=ws, save=True, **kw)
        return (out, final, *kda.kda_scan_backward(d_out, q, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu,
                                                   workspace=ws, saved=True, **kw))

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = [step(stream=s) for s in streams]
    inner = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu, stream=streams[0])  # a workspace of the stream's own
    torch.cuda.synchronize()
    for got in runs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(inner[0], want[0]) and torch.equal(inner[1], want[1])

    ws = torch.zeros(kda.scan_workspace_bytes(277, 2, H, training=True), dtype=torch.uint8, device=cuda_device)
    x = q.clone()
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out, final = kda.kda_scan(x, k, v, g, beta, state, cu_seqlens=cu, workspace=ws, save=True)
            res = (out, final, *kda.kda_scan_backward(d_out, x, k, v, g, beta, state, d_final_state=d_final, cu_seqlens=cu,
                                                      workspace=ws, saved=True))
        graphs.append((gr, res))
    for q2 in (q, q.flip(0).contiguous()):
        x.copy_(q2)
        for gr, _ in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], graphs[1][1]))
        fresh, _ = kda.kda_scan(q2, k, v, g, beta, state, cu_seqlens=cu)
        assert torch.equal(graphs[0][1][0], fresh)
    assert kda.scan_error(ws) == 0


def test_scan_two_calls_at_once(cuda_device):
    """A captured training step replayed on one stream beside an eager one on another, each with its workspace."""
    def make(lens, H, seed):
        x = inputs(lens, H, seed=seed)
        ws = torch.zeros(kda.scan_workspace_bytes(sum(lens), len(lens), H, training=True), dtype=torch.uint8, device="cuda")
        return x[:5], x[5], ws

    def step(x, cu, ws):
        out, final = kda.kda_scan(*x, cu_seqlens=cu, workspace=ws, save=True)
        return [out, final, *kda.kda_scan_backward(out, *x, cu_seqlens=cu, workspace=ws, saved=True)]

    a, b = make([700, 64, 1, 2000], 8, 21), make([333] * 30, 8, 22)
    want_a, want_b = step(*a), step(*b)
    torch.cuda.synchronize()
    one, two, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got_a = step(*a)
    for _ in range(5):
        with torch.cuda.stream(one):
            graph.replay()
        with torch.cuda.stream(two):
            got_b = step(*b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got_a + got_b, want_a + want_b))
    assert kda.scan_error(a[2]) == kda.scan_error(b[2]) == 0


def test_scan_workspace_contents_do_not_matter(cuda_device):
    q, k, v, g, beta, cu = inputs([100, 3], 2, seed=111)
    want = kda.kda_scan(q, k, v, g, beta, cu_seqlens=cu)
    ws = torch.full((kda.scan_workspace_bytes(103, 2, 2),), 255, dtype=torch.uint8, device=cuda_device)  # NaN in every type
    got = kda.kda_scan(q, k, v, g, beta, cu_seqlens=cu, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.slow
def test_scan_offsets_beyond_32_bits(cuda_device):
    """Rows 2^25 elements apart: the last ones lie 2^32 elements behind the first."""
    T, H, stride = 140, 1, 1 << 25
    q, k, v, g, beta, cu = inputs([T], H, seed=121)
    want = kda.kda_scan(q, k, v, g, beta, cu_seqlens=cu)
    buf = torch.empty(T * stride, dtype=torch.bfloat16, device=cuda_device).view(T, stride)
    views = [buf[:, i * 128:(i + 1) * 128].unflatten(-1, (H, 128)) for i in range(4)]
    for dst, src in zip(views, (q, k, v)):
        dst.copy_(src)
    got = kda.kda_scan(*views[:3], g, beta, cu_seqlens=cu, out=views[3])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_scan_long_sequence_and_prefill_agree(cuda_device):
    """Many chunks at a layer's decays, against the prefill (another algorithm, fp32 throughout) within both tolerances."""
    T, H = 2000, 4
    q, k, v, g, beta, cu = inputs([T], H, "mild", seed=131)
    state = states(1, H, 3)
    out, final = kda.kda_scan(q, k, v, g, beta, state, cu_seqlens=cu)
    pool = state.clone()
    out2 = kda.kda_prefill(*(x[None] for x in (q, k, v, g, beta)), pool, torch.zeros(1, dtype=torch.int32, device=cuda_device))
    # the prefill's documented accuracy: states 1e-5, outputs one bf16 step
    ref.check(final, pool, ref.SCAN_REL + 1e-5, "state")
    ref.check(out, out2[0], ref.SCAN_REL + 1e-5, "out", 4 * ref.BF16_HALF_STEP)


# ------------------------------------------------------------------------------------------------ refusals on the GPU
def test_binding_refusals(cuda_device):
    q, k, v, g, beta, cu = inputs([10], 2)
    call = kda.kda_scan
    with pytest.raises(TypeError):
        call(q.float(), k, v, g, beta, cu_seqlens=cu)
    with pytest.raises(TypeError):
        call(q, k, v, g.bfloat16(), beta, cu_seqlens=cu)
    with pytest.raises(TypeError):
        call(q, k, v, g, beta, cu_seqlens=cu.long())
    with pytest.raises(ValueError):
        call(q, k[:9], v, g, beta, cu_seqlens=cu)
    with pytest.raises(ValueError):
        call(q, k, v, g, beta, torch.zeros(2, 2, K, V, device=cuda_device), cu_seqlens=cu)
    with pytest.raises(TypeError):
        call(q, k, v, g, beta, torch.zeros(1, 2, K, V, device=cuda_device).transpose(2, 3), cu_seqlens=cu)
    with pytest.raises(ValueError):
        call(q, k, v, g, beta, cu_seqlens=cu, slot_idx=torch.zeros(1, dtype=torch.int32, device=cuda_device))
    with pytest.raises(ValueError):
        call(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, g, beta, cu_seqlens=cu)  # rows not dense
    with pytest.raises(ValueError):
        call(q, k, v, g, beta)  # without cu_seqlens a dense batch
    with pytest.raises(kda.KdaError):
        call(q[..., :64].contiguous(), k[..., :64].contiguous(), v, g[..., :64].contiguous(), beta, cu_seqlens=cu,
             workspace=torch.empty(1 << 20, dtype=torch.uint8, device=cuda_device))
    with pytest.raises(kda.KdaError):
        call(q, k, v, g, beta, cu_seqlens=cu, workspace=torch.empty(64, dtype=torch.uint8, device=cuda_device))
    with pytest.raises(kda.KdaError):
        call(q, k, v, g, beta, cu_seqlens=cu, out=v)
    with pytest.raises(TypeError):
        kda.kda_scan_backward(v.float(), q, k, v, g, beta, cu_seqlens=cu)
