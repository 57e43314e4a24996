"""The operators measured beside the layers: low-rank adapters of many requests at once added to a shared
projection's output, rotary positions with several axes applied to normalised q and k, and the rotary tables
that the fused q / k / v projection reads.

`run` computes them in plain torch operations, or with `own` through the library's calls.

Formulas.
  adapters  out[m] = y[m] + sum_j w[s, j] B[id(s, j)] (A[id(s, j)] x[m]) for every row m of request s; id -1 adds
            nothing; rows of no request (behind the last one) keep y.
  rope      x / sqrt(mean(x^2) + eps) * weight per head of q and k, then pair i of token m rotated by
            position[m, axis(i)] * theta^(-2 i_axis / d_axis).
  tables    cos and sin of those angles, pair-major [pairs, tokens].
"""

import random

import numpy as np
import torch

own = False

THETA = 10000.0
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _adapters(name, rows, requests, k, n, rank, slots, adapters, tail=0):
    c = {"op": "adapters", "rows": rows, "requests": requests, "k": k, "n": n, "rank": rank, "slots": slots,
         "adapters": adapters, "tail": tail}
    return dict(c, name=name) if name else c


def _rope(name, rows, batch, q_heads, k_heads, head_dim, axes, half, fractional):
    c = {"op": "rope", "rows": rows, "batch": batch, "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim,
         "axes": axes, "half": half, "fractional": fractional}
    return dict(c, name=name) if name else c


def _tables(name, rows, batch, head_dim, axes, fractional):
    c = {"op": "tables", "rows": rows, "batch": batch, "head_dim": head_dim, "axes": axes, "fractional": fractional}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the adaptive normalisation of one request: one conditioning vector, one adapter (latency)
        _adapters("adapters_adaln_1", 1, 1, 2560, 15360, 16, 1, 8),
        # the same layer for a full batch: a row per request, 24 adapters among 64 requests (weight bandwidth)
        _adapters("adapters_adaln_64", 64, 64, 2560, 15360, 64, 1, 24),
        # text tokens of 32 requests of uneven, odd lengths, three padding rows behind the last
        _adapters("adapters_text_32", 2500, 32, 2560, 7680, 32, 1, 12, tail=3),
        # the q / k / v projection of one image with two adapters stacked (style and subject)
        _adapters("adapters_qkv_image", 4608, 1, 2560, 7680, 32, 2, 4),
        # the MLP's down projection, four images at ragged resolutions, rank 128
        _adapters("adapters_down_ragged", 9001, 4, 10240, 2560, 128, 1, 4),
        # the MLP's up projection over a long sequence (video), four requests, two adapters each
        _adapters("adapters_up_video", 18432, 4, 2560, 10240, 64, 2, 6),
        # q and k of a short text-only pass
        _rope("rope_text_77", 77, 1, 20, 20, 128, "16,56,56", False, False),
        # an image with its text tokens, two guidance branches sharing the positions
        _rope("rope_image_9216", 9216, 2, 20, 20, 128, "16,56,56", False, False),
        # a long video, rotated as halves, grouped k heads, positions scaled to fractions
        _rope("rope_video_33001", 33001, 1, 24, 8, 96, "24,36,36", True, True),
        # the tables of one image
        _tables("tables_image_4608", 4608, 1, 128, "16,56,56", False),
        # the tables of a long video
        _tables("tables_video_131075", 131075, 1, 128, "44,42,42", True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "rope", "tables"])
    if op == "adapters":
        slots = rng.choice([1, 1, 2, 4])
        rank = rng.choice([r for r in (16, 32, 48, 64, 128) if r * slots <= 128])
        k, n = 64 * _log(rng, 16, 160), 64 * _log(rng, 16, 240)
        kind = rng.choice(["single", "text", "image"])
        if kind == "single":                      # a row per request
            requests = _log(rng, 1, 128)
            rows = requests
        elif kind == "text":
            requests = _log(rng, 2, 48)
            rows = requests * rng.randint(9, 200) + rng.randint(0, 7)
        else:
            requests = rng.randint(1, 6)
            rows = _log(rng, 700, 18432)
        # no dearer than the largest listed case
        rows = max(1, min(rows, 18432 * (2560 + 10240 + 10240) // (k + 2 * n),
                          18432 * 128 * (2560 + 10240) // (rank * slots * (k + n))))
        requests = min(requests, rows)
        return _adapters(None, rows, requests, k, n, rank, slots, rng.randint(2, 32),
                         rng.choice([0, 0, rng.randint(1, 5)]) if rows > 16 else 0)
    head_dim, axes = rng.choice([(64, "16,24,24"), (128, "16,56,56"), (128, "44,42,42"), (96, "24,36,36"),
                                 (128, "64,64"), (80, "16,32,32"), (256, "32,64,64")])
    batch = rng.choice([1, 1, 2])
    if op == "rope":
        k_heads = rng.choice([4, 8, 16, 20])
        q_heads = k_heads * rng.choice([1, 1, 2, 3])
        most = max(64, min(33001, 33001 * (24 + 8) * 96 // ((q_heads + k_heads) * head_dim)))
        return _rope(None, batch * _log(rng, 16, most // batch), batch, q_heads, k_heads, head_dim, axes,
                     rng.random() < 0.5, rng.random() < 0.3)
    return _tables(None, batch * _log(rng, 64, 131075 * 128 // max(128, head_dim) // batch), batch, head_dim, axes,
                   rng.random() < 0.3)


def _offsets(case):
    """Row offsets of the requests: a row each, or uneven lengths."""
    s, covered = case["requests"], case["rows"] - case["tail"]
    w = np.ones(s) if s >= covered else 1.0 + (7 * np.arange(s)) % 5
    return [0] + [int(v) for v in np.round(covered * np.cumsum(w) / w.sum())]


def _ids(case):
    """Adapter of each request and slot; every fifth request has none in its first slot."""
    s, j = case["requests"], case["slots"]
    ids = np.arange(s * j).reshape(s, j) % case["adapters"]
    ids[4::5, 0] = -1
    return ids.astype(np.int32)


def _widths(case):
    return [int(v) for v in case["axes"].split(",")]


# ---------------------------------------------------------------- inputs

def _positions(case, seed, device):
    """Rows of (time, height, width) -- or (height, width) -- positions: 64 text tokens at the origin, then a grid;
    the time (or the height) starts at an offset of the seed's, as in a window of a long video."""
    p = case["rows"] // case["batch"]
    axes = len(_widths(case))
    text = min(64, p // 4)
    i = torch.arange(p - text, device=device)
    side = 96
    cols = [i // (side * side), (i // side) % side, i % side] if axes == 3 else [i // side, i % side]
    pos = torch.stack(cols, 1)
    pos[:, 0] += random.Random(seed).randint(0, 30000)
    pos = torch.cat([torch.zeros((text, axes), dtype=pos.dtype, device=device), pos])
    return (pos.float() * 0.8125).contiguous() if case["fractional"] else pos.to(torch.int32).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(torch.bfloat16)

    if case["op"] == "adapters":
        m, k, n, r = case["rows"], case["k"], case["n"], case["rank"]
        offsets, ids = _offsets(case), _ids(case)
        weights = np.random.default_rng(seed).uniform(0.25, 1.25, ids.shape).astype(np.float32)
        x = normal(m, k)
        x[:, :: 97] *= 8                          # a few strong channels, as activations have
        st = {"case": case, "x": x, "y": normal(m, n), "a": normal(case["adapters"], r, k, scale=k ** -0.5),
              "b": normal(case["adapters"], n, r, scale=0.2 * r ** -0.5),
              "offsets": torch.tensor(offsets, device=dev), "ids": torch.from_numpy(ids).to(dev),
              "weights": torch.from_numpy(weights).to(dev), "longest": int(np.diff(offsets).max())}
        if own:                                   # the batch's plan, kept over all layers and steps
            import bit_diffusion_transformer_act_b200 as P
            st["plan"] = P.LoraPlan(offsets, ids, weights, m, case["adapters"], device=dev)
        return st
    st = {"case": case, "pos": _positions(case, seed, dev), "widths": _widths(case)}
    if case["op"] == "rope":
        m, hq, hk, d = case["rows"], case["q_heads"], case["k_heads"], case["head_dim"]
        qkv = normal(m, (hq + 2 * hk) * d)        # the projection's packed output
        st["q"] = qkv[:, : hq * d].view(m, hq, d)
        st["k"] = qkv[:, hq * d:(hq + hk) * d].view(m, hk, d)
        st["wq"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16)
        st["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16)
    return st


# ---------------------------------------------------------------- one pass

def _plain_adapters(x, y, a, b, offsets, ids, weights, longest):
    s, j = ids.shape
    # the requests' rows padded to the longest: [s, longest]
    row = offsets[:-1, None] + torch.arange(longest, device=x.device)
    real = row < offsets[1:, None]
    row = torch.where(real, row, offsets[:-1, None].clamp(max=x.shape[0] - 1))
    at = ids.clamp(min=0).long()
    w = torch.where(ids >= 0, weights, 0.0)[:, None] * real[:, :, None]
    u = torch.matmul(x[row].float(), a[at].float().flatten(1, 2).transpose(1, 2))          # [s, longest, j r]
    u = u * w.repeat_interleave(a.shape[1], 2)
    d = torch.matmul(u, b[at].float().permute(0, 1, 3, 2).flatten(1, 2))                   # [s, longest, n]
    return y.float().index_add_(0, row.flatten(), d.flatten(0, 1)).to(torch.bfloat16)   # padding rows add zeros


def _angles(pos, widths, rows, pairs):
    """[rows, pairs] in 64 bits: positions may be far."""
    freq = torch.cat([THETA ** (-torch.arange(0, d, 2, device=pos.device, dtype=torch.float64) / d) for d in widths])
    axis = torch.repeat_interleave(torch.arange(len(widths), device=pos.device),
                                   torch.tensor([d // 2 for d in widths], device=pos.device))
    ang = pos.double()[:, axis] * freq
    ang = torch.nn.functional.pad(ang, (0, pairs - ang.shape[1]))
    return ang.repeat(rows // pos.shape[0], 1)


def _plain_rotate(x, w, cos, sin, half, rot):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    c, s = cos[:, None, : rot // 2], sin[:, None, : rot // 2]
    x0, x1 = (x[..., : rot // 2], x[..., rot // 2: rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
    y0, y1 = x0 * c - x1 * s, x0 * s + x1 * c
    turned = torch.cat([y0, y1], -1) if half else torch.stack([y0, y1], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1).to(torch.bfloat16)


def run(st):
    case = st["case"]
    if own:
        import bit_diffusion_transformer_act_b200 as P
        if case["op"] == "adapters":
            return P.svdq_lora_add(st["x"], st["y"], st["a"], st["b"], st["plan"])
        if case["op"] == "rope":
            return P.svdq_qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], EPS, st["pos"], st["widths"], THETA,
                                       pairing="half" if case["half"] else "interleaved")
        return P.svdq_rope_axes_tables(st["pos"], st["widths"], THETA, case["head_dim"], case["rows"])
    if case["op"] == "adapters":
        return _plain_adapters(st["x"], st["y"], st["a"], st["b"], st["offsets"], st["ids"], st["weights"],
                               st["longest"])
    ang = _angles(st["pos"], st["widths"], case["rows"], case["head_dim"] // 2)
    cos, sin = ang.cos().float(), ang.sin().float()
    if case["op"] == "tables":
        return cos.t().contiguous(), sin.t().contiguous()
    rot = sum(st["widths"])
    return (_plain_rotate(st["q"], st["wq"], cos, sin, case["half"], rot),
            _plain_rotate(st["k"], st["wk"], cos, sin, case["half"], rot))


# ---------------------------------------------------------------- work and exact values

def work(case):
    if case["op"] == "adapters":
        m, k, n, jr = case["rows"], case["k"], case["n"], case["rank"] * case["slots"]
        lens, ids = np.diff(_offsets(case)), _ids(case)
        has = (ids >= 0) & (lens[:, None] > 0)
        busy = int(lens[has.any(1)].sum())        # rows that an adapter touches
        used = len(np.unique(ids[has]))
        per_slot = int((lens[:, None] * has).sum())
        return {"bytes": 2 * (busy * k + 2 * m * n + used * case["rank"] * (k + n)),
                "flops": 2 * per_slot * case["rank"] * (k + n)}
    p, axes, d = case["rows"] // case["batch"], len(_widths(case)), case["head_dim"]
    if case["op"] == "rope":
        v = case["rows"] * (case["q_heads"] + case["k_heads"]) * d
        return {"bytes": 2 * 2 * v + 4 * p * axes + 2 * 2 * d, "flops": 7 * v}
    return {"bytes": 4 * p * axes + 4 * case["rows"] * d, "flops": 20 * case["rows"] * d // 2}


def exact(case, seed):
    """The definition in 64 bits: request by request, axis by axis."""
    st = prepare(case, seed)
    if case["op"] == "adapters":
        x, a, b = st["x"].double(), st["a"].double(), st["b"].double()
        out = st["y"].double()
        ids, w, off = _ids(case), st["weights"].cpu().numpy(), _offsets(case)
        for s in range(case["requests"]):
            for j in range(case["slots"]):
                if ids[s, j] >= 0 and off[s + 1] > off[s]:
                    low = x[off[s]:off[s + 1]] @ a[ids[s, j]].T
                    out[off[s]:off[s + 1]] += float(w[s, j]) * (low @ b[ids[s, j]].T)
        return out
    pos = st["pos"].double().repeat(case["batch"], 1)
    cos = torch.ones((case["rows"], case["head_dim"] // 2), dtype=torch.float64, device=pos.device)
    sin = torch.zeros_like(cos)
    at = 0
    for axis, d in enumerate(st["widths"]):
        for i in range(d // 2):
            ang = pos[:, axis] * THETA ** (-2.0 * i / d)
            cos[:, at], sin[:, at] = torch.cos(ang), torch.sin(ang)
            at += 1
    if case["op"] == "tables":
        return cos.T.contiguous(), sin.T.contiguous()
    outs = []
    for x, w in ((st["q"].double(), st["wq"].double()), (st["k"].double(), st["wk"].double())):
        x = x / torch.sqrt(torch.mean(x * x, dim=-1, keepdim=True) + EPS) * w
        y = x.clone()
        for i in range(at):
            lo, hi = (i, i + at) if case["half"] else (2 * i, 2 * i + 1)
            c, s = cos[:, i, None], sin[:, i, None]
            y[..., lo] = x[..., lo] * c - x[..., hi] * s
            y[..., hi] = x[..., lo] * s + x[..., hi] * c
        outs.append(y)
    return tuple(outs)
