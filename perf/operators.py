"""The router's training operators and the 4-bit integer products: cases, their
plain forms in torch, and the calls a user makes of the library.

Four kinds of case:

gate    logits [T, E] -> the k experts of each token, their weights, tokens per
        expert and the balance loss ("forward"), and the gradient of both into
        the logits ("backward").
router  the router's product: logits of T tokens, and the gradients of the
        tokens and of the router's weights from given logit gradients.
linear  y = x W^T with W in 4-bit integers and a scale (and zero point) per
        group of columns.
experts the routed SwiGLU experts with such weights, T tokens of a decode batch.

A 4-bit matrix is held as the library lays it out: tiles of 16 rows x 128
columns of 1 KB; lane l = 16 q + r of a tile has 16 bytes, row r, and its dword
s holds columns 32 s + 8 q + (0..7), element i in nibble i / 2 + 4 (i % 2);
then the scales (BF16) as [row tile][group][16 rows], and the zero points
(bytes) in the same order.  Rows are padded to 16 and columns to 128 with
scales of zero.
"""

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step's projection of one token: latency counts
        dict(name="linear one token, 768x2048", kind="linear", T=1, N=768, K=2048, group=128,
             zero=False, out="f32"),
        # odd sizes: rows not a multiple of 16, columns not of 128, zero points
        dict(name="linear 5 tokens, 1000x800", kind="linear", T=5, N=1000, K=800, group=32,
             zero=True, out="f32"),
        # a decode batch's projection (width 4096 into twice 4096)
        dict(name="linear 16 tokens, 8192x4096", kind="linear", T=16, N=8192, K=4096, group=64,
             zero=True, out="bf16"),
        # the vocabulary head on one token: the largest matrix a step reads
        dict(name="linear one token, 131072x4096", kind="linear", T=1, N=131072, K=4096,
             group=128, zero=False, out="f32"),
        # one token of the layer shape of the headline decode
        dict(name="experts one token, 2048/768", kind="experts", T=1, H=2048, I=768, E=128, k=8,
             group=128, shared=False),
        # a small batch of the large layer shape, with its shared expert
        dict(name="experts 4 tokens, 4096/2048", kind="experts", T=4, H=4096, I=2048, E=256, k=6,
             group=32, shared=True),
        # the largest decode batch: most experts are chosen, several by more than one token
        dict(name="experts 64 tokens, 2048/768", kind="experts", T=64, H=2048, I=768, E=128, k=8,
             group=64, shared=False),
        # a short padded batch with renormalised weights
        dict(name="gate forward 200x128", kind="gate", dir="forward", T=200, E=128, k=8,
             renorm=True, padded=True),
        # a long batch of the large layer shape
        dict(name="gate forward 16384x256", kind="gate", dir="forward", T=16384, E=256, k=6,
             renorm=False, padded=False),
        # its gradient, at a token count off every tile size, renormalised and padded
        dict(name="gate backward 16001x256", kind="gate", dir="backward", T=16001, E=256, k=6,
             renorm=True, padded=True),
        # a training micro-batch of the headline layer shape, router in fp32
        dict(name="router 777, 2048x128", kind="router", T=777, H=2048, E=128, router="f32"),
        # a long batch of the large layer shape
        dict(name="router 16384, 4096x256", kind="router", T=16384, H=4096, E=256,
             router="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "experts", "gate", "router"])
    if kind == "linear":
        while True:
            c = dict(kind=kind, T=_log(rng, 1, 64), N=_log(rng, 64, 131072), K=_log(rng, 64, 8192),
                     group=rng.choice([32, 64, 128]), zero=rng.random() < 0.5,
                     out=rng.choice(["f32", "bf16"]))
            if c["N"] * c["K"] <= 1 << 28:
                return c
    if kind == "experts":
        while True:
            E = _log(rng, 8, 256)
            c = dict(kind=kind, T=_log(rng, 1, 64), H=32 * _log(rng, 8, 128),
                     I=32 * _log(rng, 4, 64), E=E, k=rng.randint(1, min(8, E)),
                     group=rng.choice([32, 64, 128]), shared=rng.random() < 0.5)
            if c["T"] * c["k"] * c["H"] * c["I"] <= 1 << 29 and E * c["H"] * c["I"] <= 1 << 30:
                return c
    if kind == "gate":
        while True:
            E = _log(rng, 4, 1024)
            c = dict(kind=kind, dir=rng.choice(["forward", "backward"]), T=_log(rng, 1, 32768),
                     E=E, k=rng.randint(1, min(8, E)), renorm=rng.random() < 0.5,
                     padded=rng.random() < 0.5)
            if c["T"] * E <= 16384 * 256:
                return c
    while True:
        c = dict(kind=kind, T=_log(rng, 16, 16384), H=32 * _log(rng, 8, 192),
                 E=_log(rng, 8, 512), router=rng.choice(["f32", "bf16"]))
        if c["T"] * c["H"] * c["E"] <= 1 << 33:
            return c


# ---------------------------------------------------------------------------
# 4-bit matrices
# ---------------------------------------------------------------------------
def _up(v, m):
    return (v + m - 1) // m * m


def _q4_sizes(N, K, group, zero):
    """bytes of (codes, scales, zero points) of one matrix"""
    tiles, cols = _up(N, 16) // 16, _up(K, 128)
    return tiles * cols * 8, tiles * (cols // group) * 32, tiles * (cols // group) * 16 if zero else 0


def _q4_random(gen, count, N, K, group, zero, std=0.02):
    """`count` matrices as one uint8 tensor [count, bytes]: codes of a rounded
    normal distribution around the zero point, scales near std / 2.3."""
    Np, Kp = _up(N, 16), _up(K, 128)
    G = Kp // group
    s = (std / 2.3) * (1.0 + 0.2 * torch.randn((count, Np, G), generator=gen, device=DEV)).abs()
    s = s.to(torch.bfloat16)
    s[:, N:] = 0
    s[:, :, (K + group - 1) // group:] = 0
    z = torch.full((count, Np, G), 8, dtype=torch.uint8, device=DEV)
    if zero:
        z = torch.randint(4, 12, (count, Np, G), generator=gen, device=DEV, dtype=torch.uint8)
    q = torch.randn((count, Np, Kp), generator=gen, device=DEV, dtype=torch.float16).mul_(2.3)
    q = q.view(count, Np, G, group).add_(z[..., None]).round_().clamp_(0, 15).to(torch.uint8)
    q = q.view(count, Np // 16, 16, Kp // 128, 4, 4, 8).permute(0, 1, 3, 5, 2, 4, 6)
    # the four bytes of a dword: elements (0, 2), (4, 6), (1, 3), (5, 7)
    codes = (q[..., [0, 4, 1, 5]] | (q[..., [2, 6, 3, 7]] << 4)).reshape(count, -1)
    tiled = lambda v: v.view(count, Np // 16, 16, G).transpose(2, 3).contiguous()
    parts = [codes, tiled(s).view(torch.uint8).reshape(count, -1)]
    if zero:
        parts.append(tiled(z).reshape(count, -1))
    return torch.cat(parts, 1)


def _q4_values(block, N, K, group, zero):
    """[count, N, K] fp32 values of matrices laid out as above."""
    count, Np, Kp = block.shape[0], _up(N, 16), _up(K, 128)
    nc, ns, nz = _q4_sizes(N, K, group, zero)
    b = block[:, :nc].view(count, Np // 16, Kp // 128, 4, 16, 4, 4)
    q = torch.cat([b & 15, b >> 4], -1)[..., [0, 2, 4, 6, 1, 3, 5, 7]]   # elements in order
    q = q.permute(0, 1, 4, 2, 5, 3, 6).reshape(count, Np, Kp // group, group)
    untiled = lambda v: v.view(count, Np // 16, Kp // group, 16).transpose(2, 3).reshape(
        count, Np, Kp // group, 1)
    s = untiled(block[:, nc:nc + ns].contiguous().view(torch.bfloat16)).float()
    z = untiled(block[:, nc + ns:nc + ns + nz]).float() if zero else 8.0
    return ((q.float() - z) * s).view(count, Np, Kp)[:, :N, :K]


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _tokens(gen, T, H):
    return torch.randn((T, H), generator=gen, device=DEV).to(torch.bfloat16)


def _gate_plain(z, routed, k, renorm):
    """ids, w, counts [E + 1], loss of the gate (ids -1 and w 0 where not routed)."""
    T, E = z.shape
    p = (z - z.max(1, keepdim=True).values).exp()
    p = p / p.sum(1, keepdim=True)
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    w = w * routed[:, None]
    ids = torch.where(routed[:, None], ids, -1)
    # tokens per expert (place 0 takes the ids of -1), and the tokens routed
    c = torch.zeros(E + 1, dtype=torch.int64, device=z.device)
    c.scatter_add_(0, (ids + 1).view(-1), torch.ones_like(ids).view(-1))
    n = routed.sum()
    counts = torch.cat([c[1:], n[None]]).to(torch.int32)
    S = (p * routed[:, None]).sum(0)
    loss = E * (c[1:].float() * S).sum() / (k * n.float().square()).clamp(min=1)
    return ids.to(torch.int32), w, counts, loss.view(1)


def prepare(case, seed):
    gen = _gen(seed)
    c = dict(case)
    kind = c["kind"]
    st = dict(case=c)
    if kind == "linear":
        st["x"] = _tokens(gen, c["T"], c["K"])
        st["w"] = _q4_random(gen, 1, c["N"], c["K"], c["group"], c["zero"])[0]
        if own:
            from sparse_expert_execution_amd import ops
            st["desc"] = ops.make_q4(c["N"], c["K"], group=c["group"], zero=c["zero"])
            st["y"] = torch.empty((c["T"], c["N"]), device=DEV, dtype=_TYPE[c["out"]])
    elif kind == "experts":
        T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
        st["x"] = _tokens(gen, T, H)
        z = torch.randn((T, E), generator=gen, device=DEV)
        top = torch.sort(torch.softmax(z, 1), 1, descending=True)
        st["ids"] = top.indices[:, :k].to(torch.int32).contiguous()
        st["w"] = top.values[:, :k].contiguous()
        n = E + int(c["shared"])
        pool = torch.zeros((n, _expert_bytes(H, I, c["group"])), dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 28) // (H * I))
        for e in range(0, n, step):
            m = min(step, n - e)
            b = torch.cat([_q4_random(gen, m, r, cols, c["group"], False)
                           for r, cols in ((I, H), (I, H), (H, I))], 1)
            pool[e:e + m, :b.shape[1]] = b
        st["pool"], st["shared"] = pool[:E], pool[E] if c["shared"] else None
        if own:
            from sparse_expert_execution_amd import ops
            st["desc"] = ops.make_desc(H, I, E, k, has_shared=c["shared"],
                                       wtype="int4_g%d" % c["group"])
            st["ws"] = ops.workspace(st["desc"], T, ops.MODE_DECODE)
            st["y"] = torch.empty((T, H), device=DEV)
    elif kind == "gate":
        T, E, k = c["T"], c["E"], c["k"]
        # a router's logits: a spread per token, some experts favoured
        z = torch.randn((T, E), generator=gen, device=DEV) * 1.3
        st["z"] = z + 0.5 * torch.randn((1, E), generator=gen, device=DEV)
        st["routed"] = torch.ones(T, dtype=torch.bool, device=DEV)
        if c["padded"]:
            st["routed"] = torch.rand(T, generator=gen, device=DEV) < 0.8
        if c["dir"] == "backward":
            st["ids"], st["w"], st["counts"], _ = _gate_plain(st["z"], st["routed"], k, c["renorm"])
            st["dw"] = torch.randn((T, k), generator=gen, device=DEV) * (0.3 / T)
            st["dloss"] = torch.full((1,), 0.02, device=DEV)
        if own:
            from sparse_expert_execution_amd import ops
            st["desc"] = ops.make_desc(256, 256, E, k, renorm=c["renorm"], router_wtype="f32")
            st["ws"] = ops.workspace(st["desc"], T, ops.MODE_GATE)
            if c["dir"] == "forward":
                st["mask"] = st["routed"].to(torch.uint8) if c["padded"] else None
                st["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
                st["w"] = torch.empty((T, k), device=DEV)
                st["counts"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
                st["loss"] = torch.empty(1, device=DEV)
            else:
                st["dz"] = torch.empty((T, E), device=DEV)
    else:
        T, H, E = c["T"], c["H"], c["E"]
        st["x"] = _tokens(gen, T, H)
        st["w"] = (torch.randn((E, H), generator=gen, device=DEV) * 0.02).to(_TYPE[c["router"]])
        # the gate's gradient: a few experts of a token carry most of it
        dz = torch.randn((T, E), generator=gen, device=DEV)
        st["dz"] = dz * torch.rand((T, E), generator=gen, device=DEV).pow(4) / T
        if own:
            from sparse_expert_execution_amd import ops
            st["desc"] = ops.make_desc(H, 256, E, 1, router_wtype=c["router"])
            st["ws"] = ops.workspace(st["desc"], T, ops.MODE_ROUTER_BACKWARD)
            st["z"] = torch.empty((T, E), device=DEV)
            st["dx"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
            st["dwr"] = torch.empty((E, H), device=DEV)
    return st


_TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _expert_parts(H, I, group):
    """[(offset, bytes)] of gate, up and down within an expert's block"""
    out, at = [], 0
    for r, cols in ((I, H), (I, H), (H, I)):
        n = sum(_q4_sizes(r, cols, group, False))
        out.append((at, n))
        at += n
    return out


def _expert_bytes(H, I, group):
    at, n = _expert_parts(H, I, group)[-1]
    return _up(at + n, 256)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    c = st["case"]
    if c["kind"] == "linear":
        return _linear(st, c)
    if c["kind"] == "experts":
        return _experts(st, c)
    if c["kind"] == "gate":
        return _forward(st, c) if c["dir"] == "forward" else _backward(st, c)
    return _router(st, c)


def _linear(st, c):
    if own:
        from sparse_expert_execution_amd import ops
        ops.q4_linear(st["desc"], st["x"], st["w"], st["y"])
        return st["y"]
    W = _q4_values(st["w"][None], c["N"], c["K"], c["group"], c["zero"])[0]
    return (st["x"].float() @ W.t()).to(_TYPE[c["out"]])


def _experts(st, c):
    if own:
        from sparse_expert_execution_amd import ops
        ops.decode(st["desc"], st["x"], st["ids"], st["w"], st["pool"], st["y"], st["ws"],
                   shared=st["shared"])
        return st["y"]
    T, H, I, k = c["T"], c["H"], c["I"], c["k"]
    blocks = st["pool"][st["ids"].view(-1).long()]                     # one per (token, rank)
    x = st["x"].float()
    o = _ffn(blocks, x.repeat_interleave(k, 0), c)
    y = (o.view(T, k, H) * st["w"][..., None]).sum(1)
    if c["shared"]:
        y = y + _ffn(st["shared"][None], x, c)
    return y


def _ffn(blocks, x, c):
    """SwiGLU experts, one block per row of x or one for all rows."""
    H, I, g = c["H"], c["I"], c["group"]
    at = _expert_parts(H, I, g)
    part = lambda i, n, m: _q4_values(blocks[:, at[i][0]:at[i][0] + at[i][1]], n, m, g, False)
    if blocks.shape[0] == 1:
        prod = lambda W, v: v @ W[0].t()
    else:
        prod = lambda W, v: torch.bmm(W, v[..., None])[..., 0]
    a = prod(part(0, I, H), x)
    h = a / (1 + (-a).exp()) * prod(part(1, I, H), x)
    return prod(part(2, H, I), h)


def _forward(st, c):
    if own:
        from sparse_expert_execution_amd import ops
        ops.gate(st["desc"], st["z"], st["ids"], st["w"], st["ws"], mask=st["mask"],
                 counts=st["counts"], loss=st["loss"])
        return dict(ids=st["ids"], w=st["w"], counts=st["counts"], loss=st["loss"])
    ids, w, counts, loss = _gate_plain(st["z"], st["routed"], c["k"], c["renorm"])
    return dict(ids=ids, w=w, counts=counts, loss=loss)


def _backward(st, c):
    if own:
        from sparse_expert_execution_amd import ops
        ops.gate_backward(st["desc"], st["z"], st["ids"], st["w"], st["dz"], dw=st["dw"],
                          counts=st["counts"], dloss=st["dloss"])
        return st["dz"]
    z, E, k = st["z"], c["E"], c["k"]
    p = (z - z.max(1, keepdim=True).values).exp()
    p = p / p.sum(1, keepdim=True)
    routed = st["ids"][:, :1] >= 0
    ids = st["ids"].long().clamp(min=0)
    n = st["counts"][E].float()
    b = st["dloss"] * E * st["counts"][:E].float() / (k * n.square()).clamp(min=1)
    dw = st["dw"]
    if c["renorm"]:                       # d(loss)/d(p) of w = p / sum of the chosen p
        dw = (dw - (dw * st["w"]).sum(1, keepdim=True)) / p.gather(1, ids).sum(1, keepdim=True)
    dp = b[None] + torch.zeros_like(p).scatter_(1, ids, dw)
    return p * (dp - (p * dp).sum(1, keepdim=True)) * routed


def _router(st, c):
    if own:
        from sparse_expert_execution_amd import ops
        ops.router_logits(st["desc"], st["x"], st["w"], st["z"])
        ops.router_backward(st["desc"], st["x"], st["w"], st["dz"], st["ws"], dx=st["dx"],
                            dw_router=st["dwr"])
        return dict(z=st["z"], dx=st["dx"], dw=st["dwr"])
    x, W = st["x"].float(), st["w"].float()
    return dict(z=x @ W.t(), dx=(st["dz"] @ W).to(torch.bfloat16), dw=st["dz"].t() @ x)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["kind"] == "linear":
        T, N, K, g = c["T"], c["N"], c["K"], c["group"]
        per_group = 3 if c["zero"] else 2
        return dict(bytes=N * K / 2 + N * math.ceil(K / g) * per_group + T * K * 2
                    + T * N * (4 if c["out"] == "f32" else 2), flops=2 * T * N * K)
    if c["kind"] == "experts":
        T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
        distinct = E * (1 - (1 - k / E) ** T) + int(c["shared"])
        one = 3 * H * I * (0.5 + 2 / c["group"])
        return dict(bytes=distinct * one + T * H * 6 + T * k * 8,
                    flops=6 * H * I * T * (k + int(c["shared"])))
    if c["kind"] == "gate":
        T, E, k = c["T"], c["E"], c["k"]
        if c["dir"] == "forward":
            return dict(bytes=T * E * 4 + T * k * 8 + E * 4 + T, flops=T * E * 6)
        return dict(bytes=T * E * 8 + T * k * 12 + E * 4, flops=T * E * 8)
    T, H, E = c["T"], c["H"], c["E"]
    wb = 4 if c["router"] == "f32" else 2
    return dict(bytes=T * H * 4 + T * E * 8 + E * H * (wb + 4), flops=6 * T * H * E)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _entries(block, N, K, group, zero, rows):
    """fp64 values of rows [a, b) of one matrix, each element looked up by its
    place: tile, lane, dword and nibble."""
    n = torch.arange(*rows, device=DEV)[:, None]
    k = torch.arange(K, device=DEV)[None]
    nb, G = _up(K, 128) // 128, _up(K, 128) // group
    nc, ns, _ = _q4_sizes(N, K, group, zero)
    lane = (k % 32) // 8 * 16 + n % 16
    byte = ((n // 16 * nb + k // 128) * 64 + lane) * 16 + (k % 128) // 32 * 4
    nib = (k % 8) // 2 + 4 * (k % 2)
    v = (block[byte + nib // 2].int() >> (4 * (nib % 2))) & 15
    at = (n // 16 * G + k // group) * 16 + n % 16
    scale = block[nc:nc + ns].contiguous().view(torch.bfloat16)[at].double()
    return (v.double() - (block[nc + ns + at].double() if zero else 8.0)) * scale


def _exact_product(x, block, N, K, group, zero):
    step = max(1, (1 << 26) // K)
    return torch.cat([x @ _entries(block, N, K, group, zero, (a, min(N, a + step))).t()
                      for a in range(0, N, step)], 1)


def exact(case, seed):
    c = dict(case)
    st = prepare(case, seed)
    if c["kind"] == "linear":
        return _exact_product(st["x"].double(), st["w"], c["N"], c["K"], c["group"], c["zero"])
    if c["kind"] == "experts":
        x, H, I, g = st["x"].double(), c["H"], c["I"], c["group"]
        at = _expert_parts(H, I, g)

        def ffn(block, rows):
            a = _exact_product(rows, block[at[0][0]:], I, H, g, False)
            u = _exact_product(rows, block[at[1][0]:], I, H, g, False)
            return _exact_product(a * torch.sigmoid(a) * u, block[at[2][0]:], H, I, g, False)

        y = torch.zeros((c["T"], H), dtype=torch.float64, device=DEV)
        for e in sorted(set(st["ids"].view(-1).tolist())):
            t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
            y.index_add_(0, t, st["w"][t, j].double()[:, None] * ffn(st["pool"][e], x[t]))
        return y + ffn(st["shared"], x) if c["shared"] else y
    if c["kind"] == "gate":
        z, E, k = st["z"].double(), c["E"], c["k"]
        logp = torch.log_softmax(z, 1)
        if c["dir"] == "forward":
            # an expert's rank: how many are ahead of it (larger, or equal and lower)
            ids = torch.argsort(-z, dim=1, stable=True)[:, :k]
            top = logp.gather(1, ids)
            w = torch.softmax(top, 1) if c["renorm"] else top.exp()
            live = st["routed"]
            ids = torch.where(live[:, None], ids, -1)
            f = torch.stack([(ids == e).sum() for e in range(E)])
            n = int(live.sum())
            loss = (f * logp.exp()[live].sum(0)).sum() * E / max(1, k * n * n)
            return dict(ids=ids.to(torch.int32), w=torch.where(live[:, None], w, 0.0),
                        counts=torch.cat([f, live.sum()[None]]).to(torch.int32),
                        loss=loss.view(1))
        # the gradient of sum(dw w) + dloss loss, by torch's own differentiation
        zz = z.clone().requires_grad_(True)
        lp = torch.log_softmax(zz, 1)
        ids = st["ids"].long()
        live = ids[:, 0] >= 0
        top = lp.gather(1, ids.clamp(min=0))
        w = torch.softmax(top, 1) if c["renorm"] else top.exp()
        n = max(1, int(live.sum()))
        f = st["counts"][:E].double() * (E / (k * n * n))
        total = (w * st["dw"].double())[live].sum() \
            + st["dloss"].double()[0] * (lp.exp()[live] @ f).sum()
        total.backward()
        return zz.grad
    x, W, dz = st["x"].double(), st["w"].double(), st["dz"].double()
    return dict(z=x @ W.t(), dx=dz @ W, dw=dz.t() @ x)
