"""The norm of queries and keys with the rotation, and its gradients, against the definition in 64 bits
(tests/layer_reference.py, which also derives the tolerances); and the layer's operators in a row."""
import math

import pytest
import torch

import linear_attention_recurrent_decode_b200 as kda
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def case(rows, H, HK, D, rot, norm, weights, pos64=False, far=1 << 20, seed=0):
    g = gen(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    q, k = randn(rows, H, D).bfloat16(), (3 * randn(rows, HK, D)).bfloat16()
    kw = dict(norm=norm, eps=1e-5)
    if weights:
        kw.update(q_weight=(1 + 0.3 * randn(D)).bfloat16(), k_weight=(1 + 0.3 * randn(D)).bfloat16())
    if rot:
        f, s = kda.rope_frequencies(rot, factor=4.0, trained_context=2048, device="cuda")
        pos = torch.randint(-far, far, (rows,), generator=g, device="cuda", dtype=torch.int64 if pos64 else torch.int32)
        kw.update(positions=pos, inv_freq=f, rope_scale=s)
    return q, k, kw


def reference(x, weight, kw):
    return ref.qk(x, kw["norm"], kw["eps"], weight, kw.get("positions"), kw.get("inv_freq"), kw.get("interleaved", False),
                  kw.get("rope_scale", 1.0))


def check_heads(got, want, what):
    """Each head to its own magnitude."""
    assert got.shape == want.shape and bool(torch.isfinite(got).all()), what
    want, got = want.double(), got.double()
    bound = ref.BF16_HALF_STEP * want.abs() + (1 + ref.BF16_HALF_STEP) * ref.QK_REL * want.abs().amax(-1, keepdim=True)
    over = (got - want).abs() - bound
    assert want.numel() == 0 or float(over.max()) <= 0, f"{what}: worst by {float(over.max())}"


SHAPES = [(1, 1, 1, 8, 0), (1, 1, 1, 16, 16), (3, 2, 1, 24, 16), (5, 3, 2, 32, 32), (7, 4, 1, 40, 16), (333, 4, 2, 64, 64),
          (50, 5, 3, 96, 48), (33, 2, 2, 104, 96), (129, 32, 8, 128, 128), (40, 8, 8, 128, 64), (9, 64, 64, 128, 32),
          (11, 3, 1, 256, 256), (70, 2, 2, 248, 80), (3000, 1, 1, 64, 32), (2, 1000, 7, 64, 64)]


@pytest.mark.parametrize("rows,H,HK,D,rot", SHAPES)
@pytest.mark.parametrize("norm,weights", [("none", False), ("l2", False), ("l2", True), ("rms", False), ("rms", True)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_forward_and_gradients(rows, H, HK, D, rot, norm, weights, interleaved, cuda_device):
    q, k, kw = case(rows, H, HK, D, rot, norm, weights, pos64=interleaved, seed=rows + D)
    kw["interleaved"] = interleaved
    got = kda.kda_qk_norm_rope(q, k, **kw)
    d = [torch.randn(x.shape, generator=gen(5 + i), device="cuda").bfloat16() for i, x in enumerate((q, k))]
    grads = kda.kda_qk_norm_rope_backward(*d, q, k, **kw)
    for i, (n, x) in enumerate((("q", q), ("k", k))):
        w = kw.get(n + "_weight")
        x64 = x.double().requires_grad_()
        w64 = None if w is None else w.double().requires_grad_()
        y = reference(x64, w64, kw)
        check_heads(got[i], y.detach(), n)
        want = torch.autograd.grad(y, [x64] + ([] if w is None else [w64]), d[i].double())
        # dx = inv (g w - x^ m): a difference whose terms are bounded by inv |g w|; a quarter of the heads' largest term
        # is reached by the result with margin for random signs, so QK_REL of 4 times its largest value
        check_heads(grads[i], want[0], "d" + n) if D > 24 else ref.check(grads[i], want[0], 16 * ref.QK_REL, "d" + n, ref.BF16_HALF_STEP)
        if w is None:
            assert grads[2 + i] is None
        else:
            # dw sums g x^ over rows and heads, with g the turned-back gradient (at most rope_scale sqrt(2) |dy| a term)
            inv = (x64 * x64).sum(-1, keepdim=True) / (D if norm == "rms" else 1) + kw["eps"]
            terms = (x64.detach() / inv.detach().sqrt()).abs() * kw.get("rope_scale", 1.0) * math.sqrt(2) * d[i].double().abs().amax(-1, keepdim=True)
            bound = ref.QK_REL * terms.sum((0, 1))
            assert grads[2 + i].dtype == torch.float32 and bool(((grads[2 + i].double() - want[1]).abs() <= bound).all()), f"dw{n}"


def test_qk_far_positions_and_frequencies(cuda_device):
    """The angle keeps its fraction of a turn at positions up to 2^31, either sign, int32 and int64 alike."""
    q, _, kw = case(64, 2, 1, 128, 128, "none", False, seed=1)
    for pos in (0, 1, 2 ** 20, 2 ** 31 - 1, -2 ** 31):
        kw["positions"] = torch.full((64,), pos, dtype=torch.int32, device="cuda")
        a, _ = kda.kda_qk_norm_rope(q, **kw)
        kw["positions"] = kw["positions"].long()
        b, _ = kda.kda_qk_norm_rope(q, **kw)
        assert torch.equal(a, b)
        # fp64 angles of 2^31 rad are off by 2^-22 in the reference and the kernel alike
        want = reference(q.double(), None, kw)
        ref.check(a, want, ref.QK_REL + 2.0 ** -20, f"position {pos}", ref.BF16_HALF_STEP)


@pytest.mark.parametrize("size", [2.0 ** -58, 2.0 ** 58])
@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_qk_magnitudes_at_the_stated_limits(norm, size, cuda_device):
    """Components around 2^-58 without an eps, and around 2^58: their squares' sum stays in fp32's range."""
    q, _, kw = case(40, 3, 1, 128, 64, norm, False, seed=8)
    q, kw["eps"] = q * size, 0.0
    got, _ = kda.kda_qk_norm_rope(q, **kw)
    d = torch.randn(q.shape, generator=gen(9), device="cuda").bfloat16()
    dq = kda.kda_qk_norm_rope_backward(d, None, q, **kw)[0]
    x = q.double().requires_grad_()
    y = reference(x, None, kw)
    check_heads(got, y.detach(), "q")
    check_heads(dq, torch.autograd.grad(y, x, d.double())[0], "dq")


def test_qk_zero_and_nonfinite_rows(cuda_device):
    """Zero heads stay zero (eps), an infinity or NaN stays in its head."""
    q, k, kw = case(20, 3, 2, 64, 32, "l2", True, seed=2)
    want = kda.kda_qk_norm_rope(q, k, **kw)
    q2 = q.clone()
    q2[3] = 0
    q2[5, 1, 7] = float("nan")
    q2[6, 2, 60] = float("inf")
    got = kda.kda_qk_norm_rope(q2, k, **kw)
    keep = torch.ones(20, 3, dtype=torch.bool, device=cuda_device)
    keep[3] = keep[5, 1] = keep[6, 2] = False
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1], want[1])
    assert bool((got[0][3] == 0).all()) and bool(torch.isnan(got[0][5, 1]).any())


def test_qk_strided_in_place_and_shapes(cuda_device):
    """Slices of one packed buffer in place (the values beside them untouched), batched shapes, q alone, nothing at all."""
    rows, H, HK, D = 37, 4, 2, 64
    q, k, kw = case(rows, H, HK, D, 32, "rms", True, seed=3)
    want = kda.kda_qk_norm_rope(q, k, **kw)
    packed = torch.full((rows, (H + 2 * HK) * D), 9.0, dtype=torch.bfloat16, device=cuda_device)
    qs, ks = packed[:, :H * D].unflatten(-1, (H, D)), packed[:, H * D:(H + HK) * D].unflatten(-1, (HK, D))
    qs.copy_(q)
    ks.copy_(k)
    got = kda.kda_qk_norm_rope(qs, ks, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert kda.kda_qk_norm_rope(qs, ks, q_out=qs, k_out=ks, **kw)[0] is qs
    assert torch.equal(qs, want[0]) and torch.equal(ks, want[1]) and bool((packed[:, (H + HK) * D:] == 9).all())
    d = [torch.randn(x.shape, device="cuda").bfloat16() for x in (q, k)]
    grads = kda.kda_qk_norm_rope_backward(*d, q, k, **kw)
    again = kda.kda_qk_norm_rope_backward(d[0], d[1], q, k, dq=d[0], dk=d[1], **kw)
    assert again[0] is d[0] and all(torch.equal(a, b) for a, b in zip(grads, again))
    kw4 = dict(kw, positions=kw["positions"][:36].view(4, 9))
    batched = kda.kda_qk_norm_rope(q[:36].view(4, 9, H, D), k[:36].view(4, 9, HK, D), **kw4)
    assert torch.equal(batched[0].view(36, H, D), want[0][:36]) and torch.equal(batched[1].view(36, HK, D), want[1][:36])
    kq = {n: x for n, x in kw.items() if n != "k_weight"}
    alone = kda.kda_qk_norm_rope(q, **kq)
    assert alone[1] is None and torch.equal(alone[0], want[0])
    empty = kda.kda_qk_norm_rope(q[:0], k[:0], **dict(kw, positions=kw["positions"][:0]))
    assert empty[0].shape == (0, H, D)
    g0 = kda.kda_qk_norm_rope_backward(q[:0], k[:0], q[:0], k[:0], **dict(kw, positions=kw["positions"][:0]))
    assert bool((g0[2] == 0).all()) and bool((g0[3] == 0).all())


def test_qk_streams_graphs_and_repeats(cuda_device):
    q, k, kw = case(5000, 8, 2, 128, 64, "rms", True, seed=4)
    d = [torch.randn(x.shape, device="cuda").bfloat16() for x in (q, k)]
    want = (*kda.kda_qk_norm_rope(q, k, **kw), *kda.kda_qk_norm_rope_backward(*d, q, k, **kw))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = (*kda.kda_qk_norm_rope(q, k, stream=s, **kw), *kda.kda_qk_norm_rope_backward(*d, q, k, stream=s, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(4096 * 128, dtype=torch.uint8, device=cuda_device)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = (*kda.kda_qk_norm_rope(q, k, **kw), *kda.kda_qk_norm_rope_backward(*d, q, k, workspace=ws, **kw))
        graphs.append((g, res))
    for _ in range(2):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, res in graphs:
        assert all(torch.equal(a, b) for a, b in zip(res, want))


@pytest.mark.slow
def test_qk_offsets_beyond_32_bits(cuda_device):
    rows, H, D, stride = 140, 2, 64, 1 << 25
    q, _, kw = case(rows, H, 1, D, 64, "l2", False, seed=5)
    want, _ = kda.kda_qk_norm_rope(q, **kw)
    buf = torch.empty(rows * stride, dtype=torch.bfloat16, device=cuda_device).view(rows, stride)
    x, y = (buf[:, i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(2))
    x.copy_(q)
    kda.kda_qk_norm_rope(x, q_out=y, **kw)
    assert torch.equal(y, want)


def test_qk_gradients_against_differences(cuda_device):
    q, k, kw = case(30, 2, 1, 64, 32, "rms", True, seed=6)
    d = torch.randn(30, 2, 64, generator=gen(7), device="cuda").bfloat16()
    kq = {n: x for n, x in kw.items() if n != "k_weight"}
    dq, _, dw, _ = kda.kda_qk_norm_rope_backward(d, None, q, **kq)
    x, w = q.double(), kw["q_weight"].double()
    dx, dwd = torch.randn_like(x), torch.randn_like(w)

    def loss(e):
        return float((reference(x + e * dx, w + e * dwd, kw) * d.double()).sum())

    numeric = (loss(1e-6) - loss(-1e-6)) / 2e-6
    analytic = float((dq.double() * dx).sum() + (dw.double() * dwd).sum())
    bound = float((dq.double() * dx).abs().sum()) * ref.BF16_HALF_STEP
    assert abs(numeric - analytic) <= bound + 1e-3


def test_qk_binding_refusals(cuda_device):
    q, k, kw = case(8, 2, 2, 64, 32, "l2", True, seed=7)
    for change, error in ((dict(norm="none"), ValueError), (dict(positions=None), ValueError), (dict(inv_freq=None), ValueError),
                          (dict(inv_freq=kw["inv_freq"].float()), TypeError), (dict(positions=kw["positions"].float()), TypeError),
                          (dict(positions=kw["positions"][:7]), TypeError), (dict(q_weight=kw["q_weight"].float()), TypeError),
                          (dict(inv_freq=kw["inv_freq"][:3].contiguous()), kda.KdaError), (dict(q_out=k), kda.KdaError),
                          (dict(q_out=q[:4]), ValueError)):
        with pytest.raises(error):
            kda.kda_qk_norm_rope(q, k, **dict(kw, **change))
    with pytest.raises(ValueError):
        kda.kda_qk_norm_rope(q, k[:, :, :32], **kw)
    with pytest.raises(ValueError):
        kda.kda_qk_norm_rope(q, k_weight=kw["k_weight"])
    with pytest.raises(TypeError):
        kda.kda_qk_norm_rope(q.float())


# ---------------------------------------------------------------------------------------------- the operators in a row
def test_layer_training_step(cuda_device):
    """Projection rows -> norm -> scan -> loss, and back through both gradients, against autograd in 64 bits."""
    lens, H, D = [70, 33], 2, 128
    rows, g = sum(lens), gen(11)
    packed = torch.randn(rows, 3 * H * D, generator=g, device="cuda").bfloat16()
    q, k, v = (packed[:, i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    decay = -torch.nn.functional.softplus(torch.randn(rows, H, D, generator=g, device="cuda"))
    beta = torch.sigmoid(torch.randn(rows, H, generator=g, device="cuda"))
    d_out = torch.randn(rows, H, D, generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, 70, 103], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    f, _ = kda.rope_frequencies(64, device="cuda")
    kw = dict(norm="l2", eps=1e-6, positions=pos, inv_freq=f)
    ws = torch.empty(kda.scan_workspace_bytes(rows, 2, H, training=True), dtype=torch.uint8, device="cuda")
    qn, kn = kda.kda_qk_norm_rope(q, k, **kw)
    out, _ = kda.kda_scan(qn, kn, v, decay, beta, cu_seqlens=cu, workspace=ws, save=True)
    d_packed = torch.empty_like(packed)
    dv = d_packed[:, 2 * H * D:].unflatten(-1, (H, D))
    dqn, dkn, _, dg, dbeta, _ = kda.kda_scan_backward(d_out, qn, kn, v, decay, beta, cu_seqlens=cu, workspace=ws, saved=True, dv=dv)
    dq, dk, _, _ = kda.kda_qk_norm_rope_backward(dqn, dkn, q, k, dq=d_packed[:, :H * D].unflatten(-1, (H, D)),
                                                 dk=d_packed[:, H * D:2 * H * D].unflatten(-1, (H, D)), **kw)
    x = packed.double().requires_grad_()
    q64, k64, v64 = (x[:, i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    gd, bt = decay.double().requires_grad_(), beta.double().requires_grad_()
    o, _ = ref.scan(reference(q64, None, kw), reference(k64, None, kw), v64, gd, bt, torch.zeros(2, H, D, D, dtype=torch.float64, device="cuda"),
                    [0, 70, 103], D ** -0.5)
    dx, dg64, db64 = torch.autograd.grad(o, [x, gd, bt], d_out.double())
    # q and k were rounded to bf16 once more on the way (2^-8 of each component, random signs): normwise a few 2^-9
    for name, a, b in (("out", out, o.detach()), ("d packed", d_packed, dx), ("dg", dg, dg64), ("dbeta", dbeta, db64)):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel < 6 * ref.BF16_HALF_STEP, (name, rel)


def test_layer_serving_prompt_then_decode(cuda_device):
    """Prompts through the norm and the scan into a state pool, then decode steps: the same as scanning everything."""
    lens, H, D, steps = [70, 129], 4, 128, 3
    g = gen(12)
    total = [n + steps for n in lens]
    q, k = (torch.randn(sum(total), H, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    v = torch.randn(sum(total), H, D, generator=g, device="cuda").bfloat16()
    decay = -torch.nn.functional.softplus(torch.randn(sum(total), H, D, generator=g, device="cuda"))
    beta = torch.sigmoid(torch.randn(sum(total), H, generator=g, device="cuda"))
    q, k = kda.kda_qk_norm_rope(q, k)
    cu = torch.tensor([0, total[0], sum(total)], dtype=torch.int32, device="cuda")
    want, wfinal = kda.kda_scan(q, k, v, decay, beta, cu_seqlens=cu)
    pool, slots = torch.zeros(5, H, D, D, device="cuda"), torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    prompt = torch.cat([torch.arange(lens[0]), total[0] + torch.arange(lens[1])]).cuda()
    pcu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
    out, _ = kda.kda_scan(*(x[prompt] for x in (q, k, v, decay, beta)), pool, cu_seqlens=pcu, slot_idx=slots)
    ref.check(out, want[prompt].float(), ref.SCAN_REL, "prompt", 2 * ref.BF16_HALF_STEP)
    for t in range(steps):
        at = torch.tensor([lens[0] + t, total[0] + lens[1] + t], device="cuda")
        o = kda.kda_decode(*(x[at][:, None].contiguous() for x in (q, k, v, decay, beta)), pool, slots)
        ref.check(o[:, 0], want[at].float(), ref.SCAN_REL, f"step {t}", 2 * ref.BF16_HALF_STEP)
    ref.check(pool[slots.long()], wfinal, ref.SCAN_REL, "state")
    assert bool((pool[[0, 2, 4]] == 0).all())
