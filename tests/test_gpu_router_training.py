"""The router's training operators on the GPU against the fp64 oracle.

Tolerances, derived before the first run:
 - ids, counts: exact (they are taken from the same fp32 logits).
 - w: exp of a difference of logits up to R = max - min of a row, whose
   rounding is 2^-24 R of the result, exp itself 2^-22, a sum of E terms in a
   tree of depth E / 64 + 6, a division: (R + E / 64 + 12) 2^-23 relative.
 - loss: that on p, plus a sum over tokens of T / (4 workgroups) + 64 + 8
   roundings at most: (R + E / 64 + T / 256 + 80) 2^-23 relative.
 - dlogits: per element, p (|b| + |B| + |D|) + |w dw| + |w D| times
   (R + E / 64 + 24) 2^-22 (the terms cancel, so relative to their sizes).
 - dx, dW: fp32 sums of n terms whose factors are off by at most 2^-17 (each
   of dz and an fp32 W): (2^-16 + n 2^-24) sum |a b|, dx half a BF16 step more;
   over random data the norm is off by under 3e-6: 1e-5.
"""

import numpy as np
import pytest
import torch

from helpers import bf16_to_f64
from oracle import training

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from sparse_expert_execution_amd import ops as _ops
    _ops._lib.lib()
    return _ops


def _gate(ops, z, k, renorm=False, mask=None, stats=True):
    T, E = z.shape
    desc = ops.make_desc(256, 256, E, k, renorm=renorm, router_wtype="f32")
    zd = torch.from_numpy(z).cuda()
    ids = torch.full((T + 1, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -9.0, device="cuda")
    counts = torch.full((E + 2,), -9, dtype=torch.int32, device="cuda")
    loss = torch.full((2,), -9.0, device="cuda")
    ws = ops.workspace(desc, T, ops.MODE_GATE)
    ws.fill_(0xCD)                                 # no initial contents are needed
    md = None if mask is None else torch.from_numpy(mask).cuda()
    ops.gate(desc, zd, ids[:T], w[:T], ws if stats else None, mask=md,
             counts=counts[:E + 1] if stats else None, loss=loss[:1] if stats else None)
    torch.cuda.synchronize()
    assert torch.all(ids[T] == -9) and torch.all(w[T] == -9)
    assert int(counts[E + 1]) == -9 and float(loss[1]) == -9
    return desc, zd, ids[:T], w[:T], counts[:E + 1], loss[:1]


def _range(z):
    f = np.where(np.isfinite(z), z, np.nan)
    return float(np.nanmax(f) - np.nanmin(f)) if np.any(np.isfinite(z)) else 0.0


GATE = [
    # T, E, k, renorm, masked
    (1, 1, 1, False, False), (1, 128, 8, True, False), (3, 5, 5, True, False),
    (200, 128, 8, True, True), (33, 64, 64, False, False), (1000, 65, 3, False, True),
    (1024, 256, 6, False, True), (1025, 300, 7, True, False), (77, 1024, 8, False, True),
    (40, 1000, 40, True, False), (4099, 20, 2, True, True),
]


def _logits(T, E, seed):
    rng = np.random.default_rng(seed)
    z = (rng.standard_normal((T, E)) * 1.5 + rng.standard_normal((1, E))).astype(np.float32)
    mask = (rng.random(T) < 0.7).astype(np.uint8)
    return z, mask, rng


@pytest.mark.parametrize("T,E,k,renorm,masked", GATE)
def test_gate(ops, T, E, k, renorm, masked):
    z, mask, _ = _logits(T, E, T + E + k)
    mask = mask if masked else None
    _, _, ids, w, counts, loss = _gate(ops, z, k, renorm, mask)
    r = training.gate(z, k, renorm, mask)
    assert np.array_equal(ids.cpu().numpy(), r["ids"])
    assert np.array_equal(counts.cpu().numpy(), r["counts"])
    R = _range(z)
    wt = (R + E / 64 + 12) * 2.0 ** -23
    assert np.all(np.abs(w.cpu().numpy() - r["w"]) <= wt * r["w"])
    lt = (R + E / 64 + T / 256 + 80) * 2.0 ** -23
    assert abs(float(loss) - r["loss"]) <= lt * r["loss"]
    # without statistics, and again: equal bits
    _, _, ids2, w2, _, _ = _gate(ops, z, k, renorm, mask, stats=False)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    assert torch.equal(_gate(ops, z, k, renorm, mask)[5], loss)


@pytest.mark.parametrize("T,E,k,renorm,masked", GATE)
@pytest.mark.parametrize("which", ["both", "dw", "dloss", "none"])
def test_gate_backward(ops, T, E, k, renorm, masked, which):
    z, mask, rng = _logits(T, E, T + E + k)
    desc, zd, ids, w, counts, _ = _gate(ops, z, k, renorm, mask if masked else None)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dloss = 0.3 * T                                   # of the size of dw in a token's logits
    use_dw, use_loss = which in ("both", "dw"), which in ("both", "dloss")
    dz = torch.full((T + 1, E), 3.0, device="cuda")
    ops.gate_backward(desc, zd, ids, w if use_dw else None, dz[:T],
                      dw=torch.from_numpy(dw).cuda() if use_dw else None,
                      counts=counts if use_loss else None,
                      dloss=torch.full((1,), dloss, device="cuda") if use_loss else None)
    torch.cuda.synchronize()
    assert torch.all(dz[T] == 3.0)
    r = training.gate(z, k, renorm, mask if masked else None)
    ref = training.gate_backward(z, r["ids"], renorm, dw if use_dw else None, r["counts"],
                                 float(np.float32(dloss)) if use_loss else None)
    n = max(1, r["counts"][E])
    b = np.abs(dloss * E * r["counts"][:E] / (k * n * n))[None] if use_loss else np.zeros((1, E))
    B = (r["p"] * b).sum(1, keepdims=True)
    wd = np.abs(r["w"] * dw) if use_dw else np.zeros((T, k))
    D = wd.sum(1, keepdims=True)
    size = r["p"] * (b + B + D)
    for j in range(k):
        t = np.nonzero(r["ids"][:, j] >= 0)[0]
        size[t, r["ids"][t, j]] += wd[t, j] + r["w"][t, j] * D[t, 0]
    tol = (_range(z) + E / 64 + 24) * 2.0 ** -22
    got = dz[:T].cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol * size)
    assert np.all(got[~r["routed"]] == 0)
    # into the logits' own storage
    ops.gate_backward(desc, zd, ids, w if use_dw else None, zd,
                      dw=torch.from_numpy(dw).cuda() if use_dw else None,
                      counts=counts if use_loss else None,
                      dloss=torch.full((1,), dloss, device="cuda") if use_loss else None)
    assert torch.equal(zd, dz[:T])


@pytest.mark.parametrize("E", [128, 20])
def test_gate_on_unaligned_logits(ops, E):
    """Logits and their gradient that start at any element."""
    T, k = 50, 4
    z, _, rng = _logits(T, E, 31)
    desc, zd, ids, w, counts, loss = _gate(ops, z, k)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    one = torch.ones(1, device="cuda")
    dz = torch.empty((T, E), device="cuda")
    ops.gate_backward(desc, zd, ids, w, dz, dw=dw, counts=counts, dloss=one)
    ws = ops.workspace(desc, T, ops.MODE_GATE)
    for shift in (1, 2, 3):
        buf = torch.full((2, shift + T * E + 1), -7.0, device="cuda")
        z2, dz2 = (b[shift:shift + T * E].view(T, E) for b in buf)
        z2.copy_(zd)
        ids2, w2, counts2 = torch.empty_like(ids), torch.empty_like(w), torch.empty_like(counts)
        loss2 = torch.empty_like(loss)
        ops.gate(desc, z2, ids2, w2, ws, counts=counts2, loss=loss2)
        ops.gate_backward(desc, z2, ids2, w2, dz2, dw=dw, counts=counts2, dloss=one)
        torch.cuda.synchronize()
        for a, b in ((ids, ids2), (w, w2), (counts, counts2), (loss, loss2), (dz, dz2)):
            assert torch.equal(a, b)
        assert torch.all(buf[:, :shift] == -7) and torch.all(buf[:, -1] == -7)


def test_gate_ties_and_signed_zeros(ops):
    z = np.zeros((4, 70), dtype=np.float32)
    z[1, ::2] = -0.0
    z[2, [3, 40, 69]] = 2.0
    z[3] = np.float32(-3e38)                          # the type's lowest values
    _, _, ids, w, counts, loss = _gate(ops, z, 4)
    r = training.gate(z, 4)
    assert np.array_equal(ids.cpu().numpy(), r["ids"])
    assert np.array_equal(counts.cpu().numpy(), r["counts"])
    assert np.allclose(w.cpu().numpy(), r["w"], rtol=1e-5, atol=0)


@pytest.mark.parametrize("renorm", [False, True])
def test_gate_with_experts_not_available(ops, renorm):
    """-inf logits, rows with fewer experts than k left, rows with none."""
    z, mask, rng = _logits(60, 130, 5)
    z[rng.random(z.shape) < 0.5] = -np.inf
    z[7, 2:] = -np.inf
    z[7, :2] = [1.0, 2.0]
    z[8] = -np.inf
    z[9] = -np.inf
    z[9, 129] = -np.finfo(np.float32).max
    desc, zd, ids, w, counts, loss = _gate(ops, z, 5, renorm, mask | (np.arange(60) == 7))
    m = mask | (np.arange(60) == 7)
    r = training.gate(z, 5, renorm, m)
    assert np.array_equal(ids.cpu().numpy(), r["ids"])
    assert np.array_equal(counts.cpu().numpy(), r["counts"])
    assert np.allclose(w.cpu().numpy(), r["w"], rtol=1e-5, atol=0)
    assert abs(float(loss) - r["loss"]) < 1e-5 * r["loss"]
    dz = torch.empty_like(zd)
    dw = rng.standard_normal((60, 5)).astype(np.float32)
    ops.gate_backward(desc, zd, ids, w, dz, dw=torch.from_numpy(dw).cuda(), counts=counts,
                      dloss=torch.ones(1, device="cuda"))
    torch.cuda.synchronize()
    ref = training.gate_backward(z, r["ids"], renorm, dw, r["counts"], 1.0)
    got = dz.cpu().numpy()
    assert np.all(np.isfinite(got)) and np.max(np.abs(got - ref)) < 1e-5
    assert np.all(got[np.isneginf(z)] == 0)


def test_gate_with_nothing_routed(ops):
    z, _, _ = _logits(50, 40, 1)
    desc, zd, ids, w, counts, loss = _gate(ops, z, 3, True, np.zeros(50, dtype=np.uint8))
    assert torch.all(ids == -1) and torch.all(w == 0)
    assert torch.all(counts == 0) and float(loss) == 0
    dz = torch.full_like(zd, 9)
    ops.gate_backward(desc, zd, ids, w, dz, dw=torch.ones_like(w), counts=counts,
                      dloss=torch.ones(1, device="cuda"))
    torch.cuda.synchronize()
    assert torch.all(dz == 0)


def test_gate_nan_and_inf_stay_in_their_row(ops):
    z, _, _ = _logits(40, 90, 2)
    ref = _gate(ops, z, 4)
    bad = z.copy()
    bad[3, 10] = np.nan
    bad[20, 5] = np.inf
    bad[30] = np.nan
    _, _, ids, w, counts, loss = _gate(ops, bad, 4)
    keep = [t for t in range(40) if t not in (3, 20, 30)]
    assert torch.equal(ids[keep], ref[2][keep]) and torch.equal(w[keep], ref[3][keep])
    assert torch.all(torch.isnan(w[[3, 20]])) and torch.all(ids[30] == -1)
    assert torch.all((ids >= -1) & (ids < 90)) and not torch.any(ids[3] == 10)
    assert int(ids[20, 0]) == 5 and torch.isnan(loss).all()


# -------------------------------------------------------------------- router
ROUTER = [
    # T, H, E, router
    (1, 32, 1, "bf16"), (31, 64, 8, "f32"), (33, 96, 17, "bf16"), (200, 256, 33, "f32"),
    (777, 2048, 128, "f32"), (515, 288, 130, "bf16"), (129, 512, 300, "bf16"),
    (300, 160, 1000, "f32"), (4100, 320, 256, "bf16"), (64, 4096, 256, "bf16"),
    (2048, 64, 20, "bf16"),
    (12289, 96, 200, "bf16"), (12289, 160, 256, "f32"), (12300, 64, 100, "f32"),
    (12300, 96, 101, "bf16"), (12300, 32, 40, "f32"), (12300, 224, 64, "bf16"),
    # dx and dW in one launch, with one and with two expert tiles of dW a workgroup
    (1000, 2048, 256, "f32"), (1000, 2048, 256, "bf16"), (500, 1024, 96, "bf16"),
    (1 << 20, 32, 3, "bf16"),                      # the most tokens
]


def _router_inputs(T, H, E, router, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    w = torch.from_numpy((rng.standard_normal((E, H)) * 0.02).astype(np.float32)).cuda()
    if router == "bf16":
        w = w.to(torch.bfloat16)
    dz = torch.from_numpy((rng.standard_normal((T, E)) * rng.random((T, E)) ** 4).astype(
        np.float32)).cuda()
    return x, w, dz


def _f64(t):
    return bf16_to_f64(t) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


def _close(got, ref, size, half=0.0):
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= size + half * (np.abs(ref) + size))
    assert np.linalg.norm(got - ref) <= (1e-5 + half) * np.linalg.norm(ref) + 1e-30


@pytest.mark.parametrize("T,H,E,router", ROUTER)
def test_router(ops, T, H, E, router):
    x, w, dz = _router_inputs(T, H, E, router, T + H + E)
    desc = ops.make_desc(H, 256, E, 1, router_wtype=router)
    z = torch.full((T + 1, E), 5.0, device="cuda")
    ops.router_logits(desc, x, w, z[:T])
    ws = ops.workspace(desc, T, ops.MODE_ROUTER_BACKWARD)
    ws.fill_(0xCD)
    dx = torch.full((T + 1, H), 5.0, dtype=torch.bfloat16, device="cuda")
    dwr = torch.full((E + 1, H), 5.0, device="cuda")
    ops.router_backward(desc, x, w, dz, ws, dx=dx[:T], dw_router=dwr[:E])
    torch.cuda.synchronize()
    assert torch.all(z[T] == 5) and torch.all(dx[T] == 5) and torch.all(dwr[E] == 5)
    xo, wo, dzo = _f64(x), _f64(w), _f64(dz)
    ax, aw, adz = np.abs(xo), np.abs(wo), np.abs(dzo)
    _close(z[:T].cpu().numpy(), xo @ wo.T, (2.0 ** -16 + H * 2.0 ** -24) * (ax @ aw.T))
    rx, rw = training.router_backward(xo, wo, dzo)
    _close(_f64(dx[:T]), rx, (2.0 ** -16 + E * 2.0 ** -24) * (adz @ aw), 2.0 ** -8)
    _close(dwr[:E].cpu().numpy(), rw, (2.0 ** -16 + T * 2.0 ** -24) * (adz.T @ ax))
    # one output alone, and again: equal bits
    dx2, dw2 = torch.empty_like(dx[:T]), torch.empty_like(dwr[:E])
    ops.router_backward(desc, None, w, dz, ws, dx=dx2)
    ops.router_backward(desc, x, None, dz, ws, dw_router=dw2)
    torch.cuda.synchronize()
    assert torch.equal(dx2, dx[:T]) and torch.equal(dw2, dwr[:E])


def test_router_without_tokens(ops):
    desc = ops.make_desc(64, 64, 9, 2)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((9, 64), dtype=torch.bfloat16, device="cuda")
    dz = torch.empty((0, 9), device="cuda")
    dwr = torch.full((9, 64), 3.0, device="cuda")
    ws = ops.workspace(desc, 0, ops.MODE_ROUTER_BACKWARD)
    ops.router_backward(desc, x, w, dz, ws, dx=x.clone(), dw_router=dwr)
    counts = torch.full((10,), 3, dtype=torch.int32, device="cuda")
    loss = torch.full((1,), 3.0, device="cuda")
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    ops.gate(desc, dz, ids, torch.empty((0, 2), device="cuda"), ws, counts=counts, loss=loss)
    ops.router_logits(desc, x, w, dz)
    ops.gate_backward(desc, dz, ids, None, dz)
    torch.cuda.synchronize()
    assert torch.all(dwr == 0) and torch.all(counts == 0) and float(loss) == 0


def test_router_rows_do_not_mix(ops):
    """A NaN token, or a NaN in one expert's gradient, stays where it belongs."""
    T, H, E = 70, 128, 40
    x, w, dz = _router_inputs(T, H, E, "bf16", 6)
    desc = ops.make_desc(H, 64, E, 1)
    ws = ops.workspace(desc, T, ops.MODE_ROUTER_BACKWARD)

    def run(x, dz):
        dx = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        dwr = torch.empty((E, H), device="cuda")
        ops.router_backward(desc, x, w, dz, ws, dx=dx, dw_router=dwr)
        torch.cuda.synchronize()
        return dx, dwr
    dx, dwr = run(x, dz)
    dz2 = dz.clone()
    dz2[69, 39] = float("nan")
    dx2, dwr2 = run(x, dz2)
    assert torch.equal(dx2[:69], dx[:69]) and torch.isnan(dx2[69]).all()
    assert torch.equal(dwr2[:39], dwr[:39]) and torch.isnan(dwr2[39]).all()
    x2 = x.clone()
    x2[69, 127] = float("nan")
    dx2, dwr2 = run(x2, dz)
    assert torch.equal(dx2, dx) and torch.equal(dwr2[:, :127], dwr[:, :127])


# --------------------------------------------------------------- used together
def _step(ops, desc, x, w, dw, dloss, mask, buf):
    ops.router_logits(desc, x, w, buf["z"])
    ops.gate(desc, buf["z"], buf["ids"], buf["w"], buf["gws"], mask=mask, counts=buf["counts"],
             loss=buf["loss"])
    ops.gate_backward(desc, buf["z"], buf["ids"], buf["w"], buf["dz"], dw=dw,
                      counts=buf["counts"], dloss=dloss)
    ops.router_backward(desc, x, w, buf["dz"], buf["rws"], dx=buf["dx"], dw_router=buf["dwr"])


def _buffers(ops, desc, T):
    H, E, k = desc.hidden, desc.n_experts, desc.top_k
    e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")
    return dict(z=e(T, E), ids=e(T, k, dtype=torch.int32), w=e(T, k), dz=e(T, E),
                counts=e(E + 1, dtype=torch.int32), loss=e(1), dx=e(T, H, dtype=torch.bfloat16),
                dwr=e(E, H), gws=ops.workspace(desc, T, ops.MODE_GATE),
                rws=ops.workspace(desc, T, ops.MODE_ROUTER_BACKWARD))


@pytest.mark.parametrize("renorm", [False, True])
def test_a_training_step_against_autograd_in_64_bits(ops, renorm):
    T, H, E, k = 300, 160, 24, 3
    x, w, _ = _router_inputs(T, H, E, "f32", 11)
    w = w * 5
    rng = np.random.default_rng(0)
    mask = (rng.random(T) < 0.8)
    dw = rng.standard_normal((T, k)).astype(np.float32) / T
    desc = ops.make_desc(H, 64, E, k, renorm=renorm, router_wtype="f32")
    buf = _buffers(ops, desc, T)
    _step(ops, desc, x, w, torch.from_numpy(dw).cuda(), torch.full((1,), 0.1, device="cuda"),
          torch.from_numpy(mask).cuda(), buf)
    torch.cuda.synchronize()
    xo = torch.from_numpy(_f64(x)).requires_grad_(True)
    wo = torch.from_numpy(_f64(w)).requires_grad_(True)
    p = torch.softmax(xo @ wo.T, 1)
    ids = buf["ids"].cpu().long()
    live = torch.from_numpy(mask)
    assert torch.all((ids >= 0).all(1) == live)
    g = p.gather(1, ids.clamp(min=0))
    if renorm:
        g = g / g.sum(1, keepdim=True)
    f = buf["counts"].cpu().double()
    loss = E / (k * f[E] ** 2) * (f[:E] * p[live].sum(0)).sum()
    (float(np.float32(0.1)) * loss + (g * torch.from_numpy(dw).double())[live].sum()).backward()
    assert abs(float(buf["loss"]) - float(loss)) < 1e-5 * float(loss)
    for got, ref, half in ((buf["dx"], xo.grad, 2.0 ** -8), (buf["dwr"], wo.grad, 0.0)):
        err = np.linalg.norm(_f64(got) - ref.numpy()) / np.linalg.norm(ref.numpy())
        assert err < 2e-5 + half


def test_a_training_step_in_a_graph(ops):
    """Captured once, replayed on new inputs with eager steps (buffers of their
    own) in between; every replay has the eager step's bits."""
    T, H, E, k = 600, 256, 64, 4
    desc = ops.make_desc(H, 64, E, k)
    x, w, _ = _router_inputs(T, H, E, "bf16", 3)
    dw, dloss = torch.empty((T, k), device="cuda"), torch.full((1,), 0.5, device="cuda")
    dw.normal_()
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    a, b = _buffers(ops, desc, T), _buffers(ops, desc, T)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _step(ops, desc, x, w, dw, dloss, mask, a)
    for i in range(4):
        x.copy_(_router_inputs(T, H, E, "bf16", 30 + i)[0])
        dw.normal_()
        mask[i::5] = False
        g.replay()
        _step(ops, desc, x, w, dw, dloss, mask, b)
        torch.cuda.synchronize()
        for n in ("ids", "w", "counts", "loss", "dz", "dx", "dwr"):
            assert torch.equal(a[n], b[n]), n


def test_two_streams_and_two_graphs_on_one_workspace(ops):
    """Calls at once on two streams, each with workspaces of its own, and two graphs
    that share a workspace and are replayed in turn, with eager calls between."""
    T, H, E, k = 777, 512, 128, 8
    desc = ops.make_desc(H, 256, E, k, router_wtype="f32")
    sets = []
    for seed in (51, 52):
        x, w, _ = _router_inputs(T, H, E, "f32", seed)
        b = dict(x=x, w=w, z=torch.empty((T, E), device="cuda"),
                 ids=torch.empty((T, k), dtype=torch.int32, device="cuda"),
                 gw=torch.empty((T, k), device="cuda"),
                 counts=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                 loss=torch.empty(1, device="cuda"), dz=torch.empty((T, E), device="cuda"),
                 dx=torch.empty((T, H), dtype=torch.bfloat16, device="cuda"),
                 dw=torch.empty((E, H), device="cuda"),
                 dgw=torch.randn((T, k), device="cuda"), one=torch.ones(1, device="cuda"),
                 ws=ops.workspace(desc, T, ops.MODE_GATE),
                 rws=ops.workspace(desc, T, ops.MODE_ROUTER_BACKWARD))
        sets.append(b)

    def step(b, ws, rws, stream=None):
        ops.router_logits(desc, b["x"], b["w"], b["z"], stream=stream)
        ops.gate(desc, b["z"], b["ids"], b["gw"], ws, counts=b["counts"], loss=b["loss"],
                 stream=stream)
        ops.gate_backward(desc, b["z"], b["ids"], b["gw"], b["dz"], dw=b["dgw"],
                          counts=b["counts"], dloss=b["one"], stream=stream)
        ops.router_backward(desc, b["x"], b["w"], b["dz"], rws, dx=b["dx"], dw_router=b["dw"],
                            stream=stream)
    outs = ("z", "ids", "gw", "counts", "loss", "dz", "dx", "dw")
    want = []
    for b in sets:
        step(b, b["ws"], b["rws"])
        torch.cuda.synchronize()
        want.append({n: b[n].clone() for n in outs})

    def check():
        torch.cuda.synchronize()
        for b, ref in zip(sets, want):
            for n in outs:
                assert torch.equal(b[n], ref[n]), n
                b[n].zero_()
    check()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for b, st in zip(sets, streams):
            step(b, b["ws"], b["rws"], stream=st)
    check()
    graphs = []
    for b in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(b, sets[0]["ws"], sets[0]["rws"])
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        step(sets[0], sets[0]["ws"], sets[0]["rws"])
        check()
