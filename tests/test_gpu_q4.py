"""4-bit integer matrices on the GPU against the fp64 oracle: quantiser, packer,
dense product, and the routed experts held in them.

Tolerances, derived before the first run.  A product sums, per group of G
columns, terms (16 + q) x and (16 + z) x exactly formed, in fp32; a term passes
through at most 2 G roundings in its group and K / G + 8 after it, each at most
2^-24 of the partial sum, which is at most A = sum |s| (32 + q + z) |x|: an
element is off by at most (2 G + K / G + 8) 2^-24 A.  That is the worst case;
over random data the roundings are independent: about sqrt(2 G) of them, of
2^-25 each, on partial sums some ten times the group's result (24 sqrt(G)
against 2.3 sqrt(G)), together under 5e-6 of the result's norm; NORM = 1e-5.  A BF16 output
adds half a step, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import synth
from helpers import bf16_to_f64
from oracle import formats, layer as olayer, q4 as oq4, training

pytestmark = pytest.mark.gpu

NORM = 1e-5


@pytest.fixture(scope="module")
def ops():
    from sparse_expert_execution_amd import ops as _ops
    _ops._lib.lib()
    return _ops


def _matrix(rng, N, K, group, zero, std=0.02):
    """random (q, scale bits, zeros) of a matrix"""
    G = -(-K // group)
    q = np.clip(np.rint(rng.standard_normal((N, K)) * 2.3 + 8), 0, 15).astype(np.uint8)
    s = formats.bf16_round((std / 2.3 * (1 + 0.3 * rng.uniform(-1, 1, (N, G)))).astype(np.float32))
    z = rng.integers(0, 16, (N, G)).astype(np.uint8) if zero else None
    return q, s, z


def _pack(ops, desc, q, s, z):
    N, K = q.shape
    c = np.zeros((N, (K + 1) // 2), dtype=np.uint8)
    c |= q[:, 0::2]
    c[:, :K // 2] |= q[:, 1::2] << 4
    block = torch.full((ops.q4_layout(desc)[1],), 0xEE, dtype=torch.uint8, device="cuda")
    ops.q4_pack(desc, torch.from_numpy(c).cuda(),
                torch.from_numpy(s.view(np.int16)).cuda().view(torch.bfloat16), block,
                zeros=None if z is None else torch.from_numpy(z).cuda())
    return block


def _bound(x, q, s, z, group):
    """worst-case error of every output (see the module's docstring)"""
    K = q.shape[1]
    zz = 8.0 if z is None else np.repeat(z.astype(np.float64), group, axis=1)[:, :K]
    a = (32 + q + zz) * np.repeat(np.abs(formats.bf16_decode(s)), group, axis=1)[:, :K]
    return (2 * group + K / group + 8) * 2.0 ** -24 * (np.abs(x) @ a.T)


def _check(got, ref, bound, bf16=False):
    got = got.astype(np.float64)
    half = 2.0 ** -8 if bf16 else 0.0
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= bound + half * (np.abs(ref) + bound))
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= (NORM + half) * norm + 1e-30


# ------------------------------------------------------------------- formats
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,K,group,zero", [(1, 1, 32, True), (17, 129, 128, False),
                                            (48, 800, 32, True), (33, 511, 64, False)])
def test_quantize_bit_exact(ops, N, K, group, zero, dtype):
    rng = np.random.default_rng(N + K)
    v = (rng.standard_normal((N, K + 3)) * 0.02).astype(np.float32)
    v[0, :min(K, 40)] = 0                                    # a group of zeros
    if N > 4:
        v[3] = np.abs(v[3])                                  # one sign only
        v[4] *= 1e-36
    src = torch.from_numpy(v).cuda().to(dtype)[:, :K]        # rows K + 3 apart
    desc = ops.make_q4(N, K, group=group, zero=zero)
    block = torch.full((ops.q4_layout(desc)[1] + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    ops.q4_quantize(desc, src, block)
    torch.cuda.synchronize()
    b = block.cpu().numpy()
    q, s, z = oq4.encode(src.float().cpu().numpy(), group, zero)
    assert np.array_equal(b[:-64], oq4.layout(q, s, z, group))
    assert np.all(b[-64:] == 0xA5)


@pytest.mark.parametrize("N,K,group,zero", [(1, 1, 32, True), (17, 129, 128, False),
                                            (40, 96, 64, True)])
def test_pack_bit_exact(ops, N, K, group, zero):
    q, s, z = _matrix(np.random.default_rng(7), N, K, group, zero)
    block = _pack(ops, ops.make_q4(N, K, group=group, zero=zero), q, s, z)
    torch.cuda.synchronize()
    assert np.array_equal(block.cpu().numpy(), oq4.layout(q, s, z, group))


# -------------------------------------------------------------------- linear
LINEAR = [
    # T, N, K, group, zero, bf16
    (1, 1, 1, 32, False, False), (1, 16, 128, 128, True, False), (1, 768, 2048, 128, False, False),
    (2, 17, 31, 32, True, False), (15, 100, 129, 64, False, True), (16, 1000, 800, 32, True, False),
    (17, 33, 1025, 128, True, False), (32, 64, 4096, 64, False, False),
    (33, 250, 640, 32, False, True), (64, 96, 1536, 128, True, False),
    (65, 50, 264, 64, True, False), (200, 40, 384, 32, False, False),
    (1, 40000, 256, 128, False, False), (3, 33000, 200, 32, True, True),
    (20, 8200, 136, 128, True, False), (50, 8193, 131, 64, False, True), (9, 8192, 72, 32, False, False),
    (40, 32784, 128, 64, False, False), (64, 32800, 300, 32, True, False),
]


@pytest.mark.parametrize("T,N,K,group,zero,bf16", LINEAR)
def test_linear(ops, T, N, K, group, zero, bf16):
    rng = np.random.default_rng(T * 7 + N + K)
    q, s, z = _matrix(rng, N, K, group, zero)
    desc = ops.make_q4(N, K, group=group, zero=zero)
    block = _pack(ops, desc, q, s, z)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    y = torch.full((T + 1, N), 77.0, dtype=torch.bfloat16 if bf16 else torch.float32,
                   device="cuda")
    ops.q4_linear(desc, x, block, y[:T])
    torch.cuda.synchronize()
    assert torch.all(y[T] == 77.0)
    xo = bf16_to_f64(x)
    _check(y[:T].float().cpu().numpy(), xo @ oq4.decode(q, s, z, group).T,
           _bound(xo, q, s, z, group), bf16)
    again = torch.empty_like(y[:T])
    ops.q4_linear(desc, x, block, again)
    assert torch.equal(again, y[:T])


@pytest.mark.parametrize("shift,pad_x,pad_y", [(0, 8, 4), (0, 5, 3), (1, 0, 1), (3, 13, 0)])
def test_linear_strides_and_alignment(ops, shift, pad_x, pad_y):
    T, N, K, group = 19, 45, 264, 32
    rng = np.random.default_rng(3)
    q, s, z = _matrix(rng, N, K, group, True)
    desc = ops.make_q4(N, K, group=group, zero=True)
    block = _pack(ops, desc, q, s, z)
    buf = torch.full((shift + T * (K + pad_x),), float("nan"), dtype=torch.bfloat16,
                     device="cuda")
    x = buf[shift:].view(T, K + pad_x)[:, :K]
    x.copy_(torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)))
    out = torch.full((shift + T * (N + pad_y),), 5.0, device="cuda")
    y = out[shift:].view(T, N + pad_y)[:, :N]
    ops.q4_linear(desc, x, block, y)
    torch.cuda.synchronize()
    xo = bf16_to_f64(x.contiguous())
    _check(y.cpu().numpy(), xo @ oq4.decode(q, s, z, group).T, _bound(xo, q, s, z, group))
    if pad_y:
        assert torch.all(out[shift:].view(T, N + pad_y)[:, N:] == 5.0)
    assert torch.all(out[:shift] == 5.0)


def test_linear_tokens_do_not_mix(ops):
    """NaN and infinities stay in their token's row; other rows keep their bits."""
    T, N, K = 20, 64, 384
    rng = np.random.default_rng(9)
    q, s, z = _matrix(rng, N, K, 64, False)
    desc = ops.make_q4(N, K, group=64)
    block = _pack(ops, desc, q, s, z)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    y, y2 = torch.empty((T, N), device="cuda"), torch.empty((T, N), device="cuda")
    ops.q4_linear(desc, x, block, y)
    x2 = x.clone()
    x2[3, 100] = float("nan")
    x2[17, 5] = float("inf")
    ops.q4_linear(desc, x2, block, y2)
    torch.cuda.synchronize()
    keep = [t for t in range(T) if t not in (3, 17)]
    assert torch.equal(y[keep], y2[keep])
    assert torch.all(torch.isnan(y2[[3, 17]]))


def test_linear_extreme_values(ops):
    """every code and zero point, large and tiny scales and inputs, exactly"""
    N, K, group = 16, 32, 32
    q = np.tile(np.arange(16, dtype=np.uint8)[:, None], (1, K))
    s = formats.bf16_round(np.float32(2.0) ** np.linspace(-100, 100, N).astype(np.int32)
                           .astype(np.float32)[:, None].astype(np.float32))
    desc = ops.make_q4(N, K, group=group, zero=True)
    for z0 in (0, 1, 8, 15, 240):
        z = np.full((N, 1), z0, dtype=np.uint8)
        block = _pack(ops, desc, q, s, z)
        x = torch.zeros((2, K), dtype=torch.bfloat16, device="cuda")
        x[0, 5] = 1.0
        x[1, 31] = -2.0 ** -20
        y = torch.empty((2, N), device="cuda")
        ops.q4_linear(desc, x, block, y)
        torch.cuda.synchronize()
        ref = bf16_to_f64(x) @ oq4.decode(q, s, z, group).T
        assert np.array_equal(y.cpu().numpy().astype(np.float64), ref)


def test_linear_on_a_side_stream_and_in_a_graph(ops):
    T, N, K = 2, 2048, 1024
    rng = np.random.default_rng(1)
    q, s, z = _matrix(rng, N, K, 128, False)
    desc = ops.make_q4(N, K, group=128)
    block = _pack(ops, desc, q, s, z)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((T, N), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ops.q4_linear(desc, x, block, y)
    for i in range(4):
        x.copy_(torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)))
        eager = torch.empty_like(y)
        ops.q4_linear(desc, x, block, eager)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
        with torch.cuda.stream(side):
            ops.q4_linear(desc, x, block, eager.zero_(), stream=side)
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


# ------------------------------------------------------------------- experts
class _Layer:
    """INT4 experts in a pool, and their fp64 values (gate, up, down)."""

    def __init__(self, ops, H, I, E, k, group, shared, seed, slots=None):
        rng = np.random.default_rng(seed)
        self.desc = ops.make_desc(H, I, E, k, has_shared=shared, wtype=f"int4_g{group}")
        off, self.bytes = ops.expert_layout(self.desc)
        self.values, blocks = [], []
        for _ in range(E + int(shared)):
            b = torch.zeros(self.bytes, dtype=torch.uint8, device="cuda")
            vals = []
            for m, (N, K) in enumerate(((I, H), (I, H), (H, I))):
                q, s, z = _matrix(rng, N, K, group, False, std=0.05)
                n = oq4.sections(N, K, group, False)[3]
                d = ops.make_q4(N, K, group=group)
                assert ops.q4_layout(d)[1] == n
                b[off[2 * m]:off[2 * m] + n] = _pack(ops, d, q, s, z)
                vals.append(oq4.decode(q, s, z, group))
            self.values.append(tuple(vals))
            blocks.append(b)
        self.shared = blocks.pop() if shared else None
        self.slot_of = None
        order = list(range(E))
        if slots is not None:                       # resident experts, in that slot order
            order = slots
            t = np.full(E, -1, dtype=np.int32)
            for s, e in enumerate(slots):
                t[e] = s
            self.slot_of = torch.from_numpy(t).cuda()
        self.pool = torch.cat([blocks[e] for e in order])
        self.k, self.E, self.H = k, E, H
        self.rng = rng

    def inputs(self, T):
        x = torch.from_numpy(self.rng.standard_normal((T, self.H)).astype(np.float32)).to(
            torch.bfloat16).cuda()
        ids = np.stack([self.rng.choice(self.E, self.k, replace=False) for _ in range(T)])
        w = self.rng.uniform(0.05, 0.4, (T, self.k)).astype(np.float32)
        return x, ids.astype(np.int32), w


def _run(ops, L, x, ids, w, ws=None):
    T = x.shape[0]
    ws = ops.workspace(L.desc, T, ops.MODE_DECODE) if ws is None else ws
    y = torch.full((T + 1, L.H), float("nan"), device="cuda")
    ops.decode(L.desc, x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), L.pool, y[:T],
               ws, slot_of=L.slot_of, shared=L.shared)
    torch.cuda.synchronize()
    assert torch.all(torch.isnan(y[T]))
    assert ops.decode_status(ws) == 0
    return y[:T].cpu().numpy()


def _oracle(L, x, ids, w, include=None):
    inc = (ids >= 0) & (ids < L.E)
    if include is not None:
        inc &= include
    return olayer.combine(bf16_to_f64(x), np.where(inc, ids, 0), w.astype(np.float64), L.values,
                          shared=L.values[-1] if L.shared is not None else None, include=inc)


# h carries the gate/up product's error (under 5e-6 of the norm; SwiGLU at most
# doubles a relative error of values of order one, twice for the product) and
# the split of h, at most 2^-18; the down product adds its own: 4e-5 in all
EXPERT_TOL = 4e-5

EXPERTS = [
    # H, I, E, k, group, shared, T
    (32, 32, 1, 1, 32, False, 1), (256, 128, 8, 2, 128, False, 1), (800, 96, 20, 3, 32, True, 5),
    (512, 256, 12, 3, 64, True, 64), (96, 160, 5, 4, 128, True, 33), (2048, 768, 16, 8, 128, False, 1),
    (160, 1056, 40, 8, 64, False, 64), (1024, 64, 6, 6, 32, False, 17),
    (2048, 64, 20, 3, 64, True, 64),
    # two row tiles a down workgroup; two of them, or one, for each
    (4096, 64, 24, 4, 64, True, 64), (4096, 160, 12, 3, 32, False, 3),
    (4128, 32, 5, 2, 128, False, 40), (8192, 64, 9, 2, 32, True, 2),
]


@pytest.mark.parametrize("H,I,E,k,group,shared,T", EXPERTS)
def test_experts(ops, H, I, E, k, group, shared, T):
    L = _Layer(ops, H, I, E, k, group, shared, seed=H + I + T)
    x, ids, w = L.inputs(T)
    y = _run(ops, L, x, ids, w)
    ref = _oracle(L, x, ids, w)
    assert np.linalg.norm(y - ref) <= EXPERT_TOL * np.linalg.norm(ref)
    assert olayer.row_rel_error(y, ref) < 10 * EXPERT_TOL
    assert np.array_equal(_run(ops, L, x, ids, w), y)          # fixed order: equal bits


def test_experts_partly_resident_and_not_routed(ops):
    L = _Layer(ops, 256, 128, 10, 3, 64, True, seed=4, slots=[7, 2, 0, 9, 5])
    x, ids, w = L.inputs(30)
    ids[4] = -1                                   # not routed
    ids[5, 1] = 99                                # outside
    ids[6] = [1, 3, 4]                            # none resident
    inc = np.isin(ids, [7, 2, 0, 9, 5])
    y = _run(ops, L, x, ids, w)
    ref = _oracle(L, x, ids, w, inc)
    assert np.linalg.norm(y - ref) <= EXPERT_TOL * np.linalg.norm(ref)
    for t in (4, 6):                              # the shared expert alone
        assert np.linalg.norm(y[t] - ref[t]) <= EXPERT_TOL * np.linalg.norm(ref[t])
    L.shared = None
    L.desc.has_shared = 0
    y = _run(ops, L, x, ids, w)
    assert np.all(y[4] == 0) and np.all(y[6] == 0)


def test_experts_all_tokens_on_one_and_the_same_id_twice(ops):
    L = _Layer(ops, 256, 96, 6, 4, 32, False, seed=8)
    x, ids, w = L.inputs(64)
    ids[:, 0] = 3
    ids[10] = 3                                   # four times the same expert
    ids[11] = [2, 3, 2, 3]
    y = _run(ops, L, x, ids, w)
    ref = _oracle(L, x, ids, w)
    assert np.linalg.norm(y - ref) <= EXPERT_TOL * np.linalg.norm(ref)
    assert olayer.row_rel_error(y, ref) < 10 * EXPERT_TOL
    ids[:] = 5                                    # all 256 pairs
    y = _run(ops, L, x, ids, w)
    ref = _oracle(L, x, ids, w)
    assert np.linalg.norm(y - ref) <= EXPERT_TOL * np.linalg.norm(ref)


def test_experts_packed_from_float(ops):
    """moe_pack_expert writes the quantiser's blocks at the layout's offsets."""
    H, I, group = 160, 96, 64
    desc = ops.make_desc(H, I, 4, 2, wtype="int4_g64")
    off, n = ops.expert_layout(desc)
    rng = np.random.default_rng(2)
    mats = [rng.standard_normal(s).astype(np.float32) for s in ((I, H), (I, H), (H, I))]
    block = torch.zeros(n, dtype=torch.uint8, device="cuda")
    ops.pack_expert(desc, block, *(torch.from_numpy(m).cuda() for m in mats))
    torch.cuda.synchronize()
    b = block.cpu().numpy()
    for i, m in enumerate(mats):
        ref = oq4.layout(*oq4.encode(m, group, False), group)
        assert np.array_equal(b[off[2 * i]:off[2 * i] + ref.size], ref)


@pytest.mark.parametrize("T", [1, 3, 64])
def test_route_decode(ops, T):
    L = _Layer(ops, 256, 128, 16, 4, 128, True, seed=T)
    x, _, _ = L.inputs(T)
    wr = torch.from_numpy((L.rng.standard_normal((16, 256)) * 0.1).astype(np.float32)).to(
        torch.bfloat16).cuda()
    ids = torch.full((T, 4), -7, dtype=torch.int32, device="cuda")
    w = torch.empty((T, 4), device="cuda")
    y = torch.empty((T, 256), device="cuda")
    ws = ops.workspace(L.desc, T, ops.MODE_DECODE)
    for _ in range(2):
        ops.route_decode(L.desc, x, wr, ids, w, L.pool, y, ws, shared=L.shared)
        torch.cuda.synchronize()
        r = olayer.route(bf16_to_f64(x), bf16_to_f64(wr), 4)
        clear = r["gap"] > 1e-4
        assert np.array_equal(ids.cpu().numpy()[clear], r["ids"][clear])
        ref = _oracle(L, x, ids.cpu().numpy(), w.cpu().numpy())
        assert np.linalg.norm(y.cpu().numpy() - ref) <= EXPERT_TOL * np.linalg.norm(ref)


def test_experts_in_a_graph_beside_eager_calls(ops):
    """A captured call and eager calls on a workspace each; replays follow the
    inputs they find."""
    L = _Layer(ops, 256, 160, 12, 3, 32, True, seed=5)
    T = 7
    x, ids, w = L.inputs(T)
    xd, idd, wd = x.clone(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    y = torch.empty((T, L.H), device="cuda")
    ws = ops.workspace(L.desc, T, ops.MODE_DECODE)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.decode(L.desc, xd, idd, wd, L.pool, y, ws, shared=L.shared)
    for _ in range(4):
        x, ids, w = L.inputs(T)
        eager = _run(ops, L, x, ids, w)
        xd.copy_(x)
        idd.copy_(torch.from_numpy(ids))
        wd.copy_(torch.from_numpy(w))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(y.cpu().numpy(), eager)


def test_experts_in_a_pool_that_fills_its_allocation(ops):
    """The last expert's blocks end with the pool (153 pages of 2 MiB): the loads
    that run ahead of the last job stay inside it.  Bytes are random codes under a
    scale of 2^-10 (BF16 0x3A80) by construction of the sections."""
    H, I, E, k, T = 2048, 768, 128, 8, 64
    desc = ops.make_desc(H, I, E, k, wtype="int4_g64")
    off, n = ops.expert_layout(desc)
    assert n * E == 153 << 21
    pool = torch.randint(0, 256, (E, n), dtype=torch.uint8, device="cuda")
    ends = list(off[2::2]) + [n]
    for m in range(3):
        part = pool[:, off[2 * m + 1]:ends[m]]
        part.view(E, -1, 2)[..., 0] = 0x80
        part.view(E, -1, 2)[..., 1] = 0x3A             # 2^-10
    ids = torch.stack([torch.randperm(E, device="cuda")[:k] for _ in range(T)]).to(torch.int32)
    ids[0] = torch.arange(E - k, E)
    w = torch.rand((T, k), device="cuda")
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    ws = ops.workspace(desc, T, ops.MODE_DECODE)
    ys = []
    for _ in range(3):
        y = torch.empty((T, H), device="cuda")
        ops.decode(desc, x, ids, w, pool.view(-1), y, ws)
        torch.cuda.synchronize()
        ys.append(y)
    assert torch.isfinite(ys[0]).all() and torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_experts_of_a_large_layer_in_far_slots(ops):
    """1024 experts, more pairs than one wave lists, slots past 4 GiB of the pool.
    Every expert holds one of four blocks, so that a small layer of these four is
    the oracle."""
    H, I, E, k, T, far = 256, 1536, 1024, 8, 64, 8000
    L = _Layer(ops, H, I, 4, 4, 128, True, seed=21)
    blocks = L.pool.view(4, L.bytes)
    assert far * L.bytes > 1 << 32
    desc = ops.make_desc(H, I, E, k, has_shared=True, wtype="int4_g128")
    assert ops.expert_layout(desc)[1] == L.bytes
    pool = torch.zeros((far + E, L.bytes), dtype=torch.uint8, device="cuda")
    slots = L.rng.permutation(E) + np.where(np.arange(E) % 2, far, 0)
    slot_of = torch.from_numpy(slots.astype(np.int32)).cuda()
    for m in range(4):
        pool[slot_of[m::4].long()] = blocks[m]
    x = torch.from_numpy(L.rng.standard_normal((T, H)).astype(np.float32)).to(
        torch.bfloat16).cuda()
    ids = np.stack([L.rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int32)
    w = L.rng.uniform(0.05, 0.4, (T, k)).astype(np.float32)
    y = torch.full((T, H), float("nan"), device="cuda")
    ops.decode(desc, x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), pool.view(-1), y,
               ops.workspace(desc, T, ops.MODE_DECODE), slot_of=slot_of, shared=L.shared)
    torch.cuda.synchronize()
    small = np.zeros((T, 4))
    np.add.at(small, (np.arange(T)[:, None], ids % 4), w.astype(np.float64))
    ref = _oracle(L, x, np.tile(np.arange(4, dtype=np.int32), (T, 1)), small)
    y = y.cpu().numpy()
    assert np.linalg.norm(y - ref) <= EXPERT_TOL * np.linalg.norm(ref)
    assert olayer.row_rel_error(y, ref) < 10 * EXPERT_TOL


def test_experts_tokens_do_not_mix(ops):
    """A padded batch: a token of NaN or infinities stays in its row, also where it
    shares its experts with others."""
    L = _Layer(ops, 256, 128, 4, 2, 32, True, seed=22)
    x, ids, w = L.inputs(21)
    clean = _run(ops, L, x, ids, w)
    bad = x.clone()
    bad[3] = float("nan")
    bad[20, 7] = float("inf")
    y = _run(ops, L, bad, ids, w)
    keep = np.setdiff1d(np.arange(21), [3, 20])
    assert np.array_equal(y[keep], clean[keep])
    assert np.all(np.isnan(y[3])) and np.all(np.isnan(y[20]))


def test_linear_past_four_gibibytes(ops):
    """The last rows of a matrix whose codes pass 32 bits, against a matrix of
    these rows alone (bytes of theirs, in a block of their own)."""
    N, K, group, last = 131072, 66048, 128, 32
    desc, part = ops.make_q4(N, K, group=group), ops.make_q4(last, K, group=group)
    off, n = ops.q4_layout(desc)
    assert off[1] > 1 << 32
    q, s, z = _matrix(np.random.default_rng(23), last, K, group, False)
    small = _pack(ops, part, q, s, z)
    codes = ops.q4_layout(part)[0][1]
    block = torch.zeros(n, dtype=torch.uint8, device="cuda")
    block[off[1] - codes:off[1]] = small[:codes]
    block[n - (small.numel() - codes):] = small[codes:]
    for T in (1, 6):
        x = torch.from_numpy(np.random.default_rng(T).standard_normal((T, K)).astype(
            np.float32)).to(torch.bfloat16).cuda()
        y = torch.full((T, N), float("nan"), device="cuda")
        ops.q4_linear(desc, x, block, y)
        torch.cuda.synchronize()
        xo = bf16_to_f64(x)
        assert torch.all(y[:, :N - last] == 0)
        _check(y[:, N - last:].cpu().numpy(), xo @ oq4.decode(q, s, z, group).T,
               _bound(xo, q, s, z, group))


def test_experts_from_the_cache(ops):
    """INT4 experts through the expert cache: planned, filled, decoded."""
    H, I, E, k = 256, 96, 12, 3
    L = _Layer(ops, H, I, E, k, 32, False, seed=21)
    host = L.pool.cpu().pin_memory()
    dev = torch.empty(4 * L.bytes, dtype=torch.uint8, device="cuda")
    table = torch.empty((1, E), dtype=torch.int32, device="cuda")
    cache = ops.ExpertCache(host, 1, E, L.bytes, dev, 4, table)
    side = torch.cuda.Stream()
    ws = ops.workspace(L.desc, 1, ops.MODE_DECODE)
    for _ in range(6):
        x, ids, w = L.inputs(1)
        plan = cache.plan(0, ids[0], w[0], k)
        cache.fill(plan, side)
        y = torch.empty((1, H), device="cuda")
        ops.decode(L.desc, x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), dev, y, ws,
                   slot_of=table[0])
        cache.release(plan)
        torch.cuda.synchronize()
        ref = _oracle(L, x, ids, w)
        assert np.linalg.norm(y.cpu().numpy() - ref) <= EXPERT_TOL * np.linalg.norm(ref)


# --------------------------------------------------------------- used together
def test_a_decode_step_of_the_operators_together(ops):
    """Logits, gate with load counts over a padded batch, INT4 experts, and a
    dense 4-bit product of the layer's output."""
    H, I, E, k, T, V = 256, 128, 16, 4, 24, 500
    L = _Layer(ops, H, I, E, k, 64, True, seed=77)
    x, _, _ = L.inputs(T)
    rng = L.rng
    wr = torch.from_numpy((rng.standard_normal((E, H)) * 0.1).astype(np.float32)).to(
        torch.bfloat16).cuda()
    mask = np.ones(T, dtype=np.uint8)
    mask[20:] = 0
    logits = torch.empty((T, E), device="cuda")
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    counts = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    ops.router_logits(L.desc, x, wr, logits)
    ops.gate(L.desc, logits, ids, w, ops.workspace(L.desc, T, ops.MODE_GATE),
             mask=torch.from_numpy(mask).cuda(), counts=counts)
    y = torch.empty((T, H), device="cuda")
    ops.decode(L.desc, x, ids, w, L.pool, y, ops.workspace(L.desc, T, ops.MODE_DECODE),
               shared=L.shared)
    q, s, z = _matrix(rng, V, H, 32, True)
    d = ops.make_q4(V, H, group=32, zero=True)
    out = torch.empty((T, V), device="cuda")
    yb = y.to(torch.bfloat16)
    ops.q4_linear(d, yb, _pack(ops, d, q, s, z), out)
    torch.cuda.synchronize()
    zo = logits.cpu().numpy().astype(np.float64)
    exact = bf16_to_f64(x) @ bf16_to_f64(wr).T
    assert np.max(np.abs(zo - exact)) <= H * 2.0 ** -24 * np.max(
        np.abs(bf16_to_f64(x)) @ np.abs(bf16_to_f64(wr)).T)
    r = training.gate(zo, k, mask=mask)
    assert np.array_equal(ids.cpu().numpy(), r["ids"])
    assert np.array_equal(counts.cpu().numpy(), r["counts"]) and r["counts"][E] == 20
    ref = _oracle(L, x, r["ids"], w.cpu().numpy())
    assert np.linalg.norm(y.cpu().numpy() - ref) <= EXPERT_TOL * np.linalg.norm(ref)
    yo = bf16_to_f64(yb)
    _check(out.cpu().numpy(), yo @ oq4.decode(q, s, z, 32).T, _bound(yo, q, s, z, 32))
