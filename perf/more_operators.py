"""The training and 8-bit operators of a mixture-of-experts layer as measured cases.

Every case is one pass through one operator of combine_moe_layout_02_amd:

  ffn       the experts' gated feed-forward block in bf16: moe_expert_gemm twice; a case that trains adds
            moe_expert_gemm_backward_x and moe_expert_gemm_backward_w, twice each
  int8      the experts' product in 8-bit integers: moe_quantize_i8 of the bf16 rows, then moe_expert_gemm_i8
  dispatch  moe_dispatch_i8, then moe_dequantize_i8 of the rows that hold an entry
  combine   moe_combine_backward

With ``own`` false, run() computes the same results in elementary torch
operations; with ``own`` true it makes the library's calls.

Formulas.  Of a row r of expert e: (g, u) = x[r] W_in[e]^T, h = silu(g) * u, y[r] = h W_out[e]^T; its gradients follow
from the chain rule, the weights' as sums over the expert's rows.  An 8-bit row has the scale amax/127 and codes
round(x / scale), ties to the even code; a product is the integer sum times the row's and the channel's scale.  Of
out[t] = sum_k w[t,k] y[pos[t,k]]: d_y[pos[t,k]] = w[t,k] d_out[t], d_w[t,k] = <d_out[t], y[pos[t,k]]>, 0 where pos is -1.
"""
import math

import torch

own = False

PAD_NONE, PAD_MULTIPLE, PAD_CAPACITY = 0, 1, 2
ZIPF_S = 0.875        # exponent of the skewed routing: the hottest expert gets ~20 times the mean at 256 experts


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token through its eight experts
        dict(name="ffn token", kind="ffn", S=1, H=7168, N=1024, E=32, K=8, pad_mode=PAD_NONE, pad_rows=0, zipf=False, train=False),
        # a decode batch: about four rows per expert, the weights' bytes are the work
        dict(name="ffn decode", kind="ffn", S=128, H=7168, N=1024, E=256, K=8, pad_mode=PAD_CAPACITY, pad_rows=128, zipf=False,
             train=False),
        # a prompt through few large experts: the matrix units are the bound
        dict(name="ffn prompt", kind="ffn", S=16384, H=2048, N=1408, E=64, K=6, pad_mode=PAD_NONE, pad_rows=0, zipf=False, train=False),
        # a training step of a small layer: latency of six products
        dict(name="train small", kind="ffn", S=256, H=512, N=264, E=16, K=2, pad_mode=PAD_NONE, pad_rows=0, zipf=False, train=True),
        # a training step with skewed routing, segments padded to 128 rows
        dict(name="train skew", kind="ffn", S=4096, H=2048, N=1000, E=64, K=6, pad_mode=PAD_MULTIPLE, pad_rows=128, zipf=True,
             train=True),
        # a training step at full length
        dict(name="train prompt", kind="ffn", S=16384, H=2048, N=1408, E=64, K=6, pad_mode=PAD_NONE, pad_rows=0, zipf=False, train=True),
        # the decode batch's gate and up products in 8 bits
        dict(name="int8 decode", kind="int8", S=128, H=7168, N=1024, E=256, K=8, pad_mode=PAD_CAPACITY, pad_rows=128, zipf=False,
             act=True),
        # the prompt's down product in 8 bits
        dict(name="int8 prompt", kind="int8", S=16384, H=1408, N=2048, E=64, K=6, pad_mode=PAD_NONE, pad_rows=0, zipf=False, act=False),
        # the decode call's dispatch: fixed capacity, a few rows per expert
        dict(name="dispatch decode", kind="dispatch", S=128, H=7168, E=256, K=8, pad_mode=PAD_CAPACITY, pad_rows=128, zipf=False),
        # a prompt's dispatch with ragged segments
        dict(name="dispatch prefill", kind="dispatch", S=4096, H=7168, E=256, K=8, pad_mode=PAD_NONE, pad_rows=0, zipf=False),
        # the gradient of a small layer's combine
        dict(name="combine small", kind="combine", S=256, H=512, E=16, K=2, pad_mode=PAD_NONE, pad_rows=0, zipf=False),
        # the gradient of the prefill batch's combine, segments padded to 128 rows
        dict(name="combine prefill", kind="combine", S=4096, H=7168, E=256, K=8, pad_mode=PAD_MULTIPLE, pad_rows=128, zipf=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["ffn", "ffn", "ffn", "int8", "int8", "dispatch", "combine"])
    while True:
        E = rng.choice([1, 2, 3, 5, 8, 16, 24, 60, 64, 96, 128, 160, 256])
        K = rng.randint(1, min(E, 10))
        S = _log(rng, 1, 65536 // K)
        H = 8 * _log(rng, 16, 896)
        pad_mode = rng.choice([PAD_NONE, PAD_MULTIPLE, PAD_CAPACITY])
        pad_rows = {PAD_NONE: 0, PAD_MULTIPLE: rng.choice([16, 100, 128]), PAD_CAPACITY: max(1, 2 * S * K // E)}[pad_mode]
        c = dict(kind=kind, S=S, H=H, E=E, K=K, pad_mode=pad_mode, pad_rows=pad_rows, zipf=rng.random() < 0.3)
        if kind in ("ffn", "int8"):
            c["N"] = 8 * _log(rng, 8, 256)
        if kind == "ffn":
            c["train"] = rng.random() < 0.6
        if kind in ("int8", "dispatch"):
            c["H"] = (H + 15) // 16 * 16
        if kind == "int8":
            c["act"] = rng.random() < 0.5
        w = work(c)
        # no more than the largest listed case; and the plain form, which runs every expert at the longest segment's
        # length, has to fit the card
        if w["flops"] <= 5e12 and w["bytes"] <= 10e9 and E * min(S, (8 if c["zipf"] else 2) * (S * K // E) + 64) <= 300000:
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _routing(g, S, E, K, zipf, dev):
    """K distinct experts per token: uniform, or skewed (probability ~ (e+1)^-ZIPF_S, Gumbel-top-K)."""
    u = torch.rand((S, E), generator=g, device=dev, dtype=torch.float64).clamp_(1e-300)
    key = -torch.log((-torch.log(u)).clamp_(1e-300))
    if zipf:
        key = key - ZIPF_S * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float64))
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K].to(torch.int32).contiguous()


def _layout(idx, E, pad_mode, pad_rows):
    """Counts, offsets and maps of the expert-grouped receive buffer, as the layout defines them."""
    S, K = idx.shape
    dev, n = idx.device, S * K
    flat = idx.reshape(-1).long()
    count = torch.zeros(E, dtype=torch.int64, device=dev).scatter_add_(0, flat, torch.ones_like(flat))
    order = torch.sort(flat, stable=True).indices
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(n, device=dev) - (torch.cumsum(count, 0) - count)[flat[order]]
    if pad_mode == PAD_CAPACITY:
        placed, size = count.clamp(max=pad_rows), torch.full_like(count, pad_rows)
        rows = E * pad_rows
    elif pad_mode == PAD_MULTIPLE:
        placed, size = count, (count + pad_rows - 1) // pad_rows * pad_rows
        rows = n + E * (pad_rows - 1)
    else:
        placed, size, rows = count, count, n
    off = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    off[1:] = torch.cumsum(size, 0)
    pos = torch.where(rank < placed[flat], off[flat] + rank, -1)
    src = torch.full((rows + 1,), -1, dtype=torch.int64, device=dev)
    src[torch.where(pos >= 0, pos, rows)] = torch.arange(n, device=dev)
    i32 = torch.int32
    return dict(rows=rows, most=int(placed.max()), count=placed.to(i32), offset=off.to(i32), pos=pos.to(i32).reshape(S, K),
                src=src[:rows].to(i32).contiguous(), per_rank=placed.sum().reshape(1).to(i32),
                rank_offset=torch.stack([off[0], off[E]]).to(i32), status=torch.zeros(1, dtype=i32, device=dev))


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c, s = case, {"case": case}
    S, H, E, K = c["S"], c["H"], c["E"], c["K"]
    s["lay"] = _layout(_routing(g, S, E, K, c["zipf"], dev), E, c["pad_mode"], c["pad_rows"])
    rows = s["lay"]["rows"]

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(0.0, std, generator=g)

    def row_buffer(width):
        """Rows in the layout's order; those that hold no entry were never written."""
        x = normal(rows, width)
        x[s["lay"]["src"] < 0] = math.nan
        return x

    # result rows, one more than the receive buffer: entries that have no row go there in the plain form
    def result(width):
        return torch.zeros((rows + 1, width), dtype=torch.bfloat16, device=dev)

    if c["kind"] == "ffn":
        N = c["N"]
        s["x"], s["w_in"], s["w_out"] = row_buffer(H), normal(E, 2 * N, H, std=H ** -0.5), normal(E, H, N, std=N ** -0.5)
        s["y"] = result(H)
        if c["train"]:
            s["dy"], s["dx"] = row_buffer(H), result(H)
    elif c["kind"] == "int8":
        n = c["N"] * (2 if c["act"] else 1)
        s["x"] = row_buffer(H)
        # weights as they are kept: codes, laid out once, and a scale per channel
        s["w"] = torch.randint(-127, 128, (E, n, H), generator=g, device=dev, dtype=torch.int8)
        s["ws"] = (0.5 + torch.rand((E, n), generator=g, device=dev)) * (H ** -0.5 / 73.0)
        s["out"] = result(c["N"])
    elif c["kind"] == "dispatch":
        s["x"] = normal(S, H)
        s["w"] = torch.softmax(torch.randn((S, K), generator=g, device=dev), 1)
        s["codes"] = torch.zeros((rows, H), dtype=torch.int8, device=dev)
        s["scales"] = torch.zeros(rows, device=dev)
        s["recv_w"] = torch.zeros(rows + 1, device=dev)
        s["out"] = result(H)
    else:
        s["y"], s["d_out"] = row_buffer(H), normal(S, H)
        s["w"] = torch.softmax(torch.randn((S, K), generator=g, device=dev), 1)
        s["d_y"] = result(H)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"ffn": _own_ffn, "int8": _own_int8, "dispatch": _own_dispatch, "combine": _own_combine}[kind](state)
    return {"ffn": _plain_ffn, "int8": _plain_int8, "dispatch": _plain_dispatch, "combine": _plain_combine}[kind](state)


def _own_layout(moe, s):
    c, l = s["case"], s["lay"]
    return (moe.LayoutDesc(c["S"], c["K"], c["E"], 1, c["pad_mode"], c["pad_rows"]),
            moe.Layout(l["count"], l["per_rank"], l["offset"], l["rank_offset"], l["pos"], l["src"], l["status"]))


def _own_ffn(s):
    import combine_moe_layout_02_amd as moe
    desc, lay = _own_layout(moe, s)
    rows, x, w_in, w_out = s["lay"]["rows"], s["x"], s["w_in"], s["w_out"]
    if not s["case"]["train"]:
        h = moe.moe_expert_gemm(desc, lay, x, w_in, act=moe.MOE_ACT_SWIGLU)
        return moe.moe_expert_gemm(desc, lay, h, w_out, out=s["y"][:rows])
    pre = torch.empty((rows, w_in.shape[1]), dtype=torch.float32, device=x.device)
    h = moe.moe_expert_gemm(desc, lay, x, w_in, act=moe.MOE_ACT_SWIGLU, pre=pre)
    y = moe.moe_expert_gemm(desc, lay, h, w_out, out=s["y"][:rows])
    d_pre = moe.moe_expert_gemm_backward_x(desc, lay, s["dy"], w_out, pre=pre)
    dw_out = moe.moe_expert_gemm_backward_w(desc, lay, s["dy"], h)
    dx = moe.moe_expert_gemm_backward_x(desc, lay, d_pre, w_in, out=s["dx"][:rows])
    dw_in = moe.moe_expert_gemm_backward_w(desc, lay, d_pre, x)
    return {"y": y, "dx": dx, "dw_in": dw_in, "dw_out": dw_out}


def _own_int8(s):
    import combine_moe_layout_02_amd as moe
    desc, lay = _own_layout(moe, s)
    codes, scales = moe.moe_quantize_i8(s["x"], layout=lay)
    return moe.moe_expert_gemm_i8(desc, lay, codes, scales, s["w"], s["ws"],
                                  act=moe.MOE_ACT_SWIGLU if s["case"]["act"] else moe.MOE_ACT_NONE, out=s["out"][:s["lay"]["rows"]])


def _own_dispatch(s):
    import combine_moe_layout_02_amd as moe
    desc, lay = _own_layout(moe, s)
    rows = s["lay"]["rows"]
    codes, scales, recv_w = moe.moe_dispatch_i8(desc, lay, s["x"], s["w"], recv=s["codes"], recv_scales=s["scales"],
                                                recv_w=s["recv_w"][:rows])
    return {"rows": moe.moe_dequantize_i8(codes, scales, out=s["out"][:rows], layout=lay), "recv_w": recv_w}


def _own_combine(s):
    import combine_moe_layout_02_amd as moe
    desc, lay = _own_layout(moe, s)
    d_y, d_w = moe.moe_combine_backward(desc, lay, s["d_out"], s["y"], s["w"], d_expert_out=s["d_y"][:s["lay"]["rows"]])
    return {"d_y": d_y, "d_w": d_w}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _segments(s):
    """Row of each expert's m-th entry [E, most], and whether it has one."""
    l = s["lay"]
    at = torch.arange(l["most"], device=l["offset"].device)
    holds = at < l["count"][:, None]
    return (l["offset"][:-1, None] + at).long(), holds


def _rows_of(x, row, holds):
    """The experts' rows in fp32, [E, most, width]; zeros where an expert has no more."""
    return torch.where(holds[:, :, None], x[torch.where(holds, row, 0)].float(), 0.0)


def _store(out, v, row, holds):
    """Rows back to their places, rounded once; the buffer's last row takes those that have none."""
    out[torch.where(holds, row, out.shape[0] - 1)] = v.to(torch.bfloat16)
    return out[:-1]


def _times(x, w):
    """x [E, m, k] times w [E, n, k] over k."""
    return torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2)


def _plain_ffn(s):
    N = s["case"]["N"]
    row, holds = _segments(s)
    x, w_in, w_out = _rows_of(s["x"], row, holds), s["w_in"].float(), s["w_out"].float()
    pre = _times(x, w_in)
    g, u = pre[:, :, :N], pre[:, :, N:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    h = g * sig * u
    y = _store(s["y"], _times(h, w_out), row, holds)
    if not s["case"]["train"]:
        return y
    dy = _rows_of(s["dy"], row, holds)
    dh = torch.bmm(dy, w_out)
    d_pre = torch.cat([dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig], 2)
    dx = _store(s["dx"], torch.bmm(d_pre, w_in), row, holds)
    dw_out = torch.bmm(dy.transpose(1, 2).contiguous(), h.contiguous()).to(torch.bfloat16)
    dw_in = torch.bmm(d_pre.transpose(1, 2).contiguous(), x).to(torch.bfloat16)
    return {"y": y, "dx": dx, "dw_in": dw_in, "dw_out": dw_out}


def _quantised(x):
    """Codes (as fp32) and scales of fp32 rows of finite values."""
    scale = x.abs().amax(-1, keepdim=True) / 127.0
    return torch.where(scale > 0, torch.round(x / torch.where(scale > 0, scale, 1.0)), 0.0).clamp(-127.0, 127.0), scale


def _plain_int8(s):
    N = s["case"]["N"]
    row, holds = _segments(s)
    q, scale = _quantised(_rows_of(s["x"], row, holds))
    y = _times(q, s["w"].float()) * scale * s["ws"][:, None, :]
    if s["case"]["act"]:
        g = y[:, :, :N]
        y = g / (1.0 + torch.exp(-g)) * y[:, :, N:]
    return _store(s["out"], y, row, holds)


def _plain_dispatch(s):
    K, l = s["case"]["K"], s["lay"]
    row = torch.where(l["pos"] >= 0, l["pos"], l["rows"]).reshape(-1).long()
    q, scale = _quantised(s["x"].float())
    s["out"][row] = (q * scale).to(torch.bfloat16).repeat_interleave(K, 0)
    s["recv_w"][row] = s["w"].reshape(-1)
    return {"rows": s["out"][:-1], "recv_w": s["recv_w"][:-1]}


def _plain_combine(s):
    pos, rows = s["lay"]["pos"].long(), s["lay"]["rows"]
    got = pos >= 0
    d_out = s["d_out"].float()[:, None, :]
    y = torch.where(got[:, :, None], s["y"][pos.clamp(min=0)].float(), 0.0)
    d_w = (d_out * y).sum(2)
    s["d_y"][torch.where(got, pos, rows)] = (s["w"][:, :, None] * d_out).to(torch.bfloat16)
    return {"d_y": s["d_y"][:-1], "d_w": d_w}


# ---------------------------------------------------------------------------
# what a pass cannot do without, and what it should give
# ---------------------------------------------------------------------------

def work(case):
    c = case
    S, H, E, K = c["S"], c["H"], c["E"], c["K"]
    rows = min(S * K, E * c["pad_rows"]) if c["pad_mode"] == PAD_CAPACITY else S * K
    touched = E * (1.0 - (1.0 - K / E) ** S)   # experts that any token picked, on average
    if c["kind"] == "ffn":
        product, weights = 2 * rows * c["N"] * H, 6 * c["N"] * H
        if not c["train"]:
            return {"bytes": 4 * rows * H + touched * weights, "flops": 3 * product}
        return {"bytes": 8 * rows * H + (touched + E) * weights, "flops": 9 * product}
    if c["kind"] == "int8":
        n = c["N"] * (2 if c["act"] else 1)
        return {"bytes": 2 * rows * (H + c["N"]) + touched * n * (H + 4), "flops": 2 * rows * n * H}
    if c["kind"] == "dispatch":
        # the rows go out in 8 bits, come back and leave as the values they stand for
        return {"bytes": 2 * S * H + rows * (2 * (H + 4) + 2 * H) + 12 * S * K, "flops": 3 * S * H + rows * H}
    return {"bytes": 2 * S * H + 4 * rows * H + 12 * S * K, "flops": 3 * rows * H}


def exact(case, seed):
    s = prepare(case, seed)
    return {"ffn": _exact_ffn, "int8": _exact_int8, "dispatch": _exact_dispatch, "combine": _exact_combine}[case["kind"]](s)


def _exact_experts(s):
    """(expert, its rows as a slice) for every expert with a row."""
    off, cnt = s["lay"]["offset"].tolist(), s["lay"]["count"].tolist()
    return [(e, slice(off[e], off[e] + cnt[e])) for e in range(s["case"]["E"]) if cnt[e]]


def _exact_ffn(s):
    """The block in 64 bits, expert by expert, differentiated by autograd."""
    c, rows, train = s["case"], s["lay"]["rows"], s["case"]["train"]
    dev = s["x"].device
    y = torch.zeros((rows, c["H"]), dtype=torch.float64, device=dev)
    out = {"y": y, "dx": torch.zeros_like(y), "dw_in": torch.zeros(s["w_in"].shape, device=dev),
           "dw_out": torch.zeros(s["w_out"].shape, device=dev)} if train else y
    for e, r in _exact_experts(s):
        x, w1, w2 = (t.double().requires_grad_(train) for t in (s["x"][r], s["w_in"][e], s["w_out"][e]))
        gate, up = (x @ w1.t()).chunk(2, 1)
        v = (torch.nn.functional.silu(gate) * up) @ w2.t()
        y[r] = v.detach()
        if train:
            out["dx"][r], out["dw_in"][e], out["dw_out"][e] = torch.autograd.grad(v, (x, w1, w2), s["dy"][r].double())
    return out


def _exact_codes(x):
    top = x.double().abs().amax(1, keepdim=True)
    return torch.round(x.double() * 127.0 / torch.where(top > 0, top, 1.0)), top / 127.0


def _exact_int8(s):
    c = s["case"]
    out = torch.zeros((s["lay"]["rows"], c["N"]), dtype=torch.float64, device=s["x"].device)
    for e, r in _exact_experts(s):
        q, scale = _exact_codes(s["x"][r])
        v = (q @ s["w"][e].double().t()) * (scale * s["ws"][e].double())
        out[r] = torch.nn.functional.silu(v[:, :c["N"]]) * v[:, c["N"]:] if c["act"] else v
    return out


def _exact_dispatch(s):
    src, K = s["lay"]["src"].long(), s["case"]["K"]
    q, scale = _exact_codes(s["x"])
    held = torch.nonzero(src >= 0).reshape(-1)
    rows = torch.zeros((src.numel(), s["x"].shape[1]), device=src.device)
    rows[held] = (q * scale).float()[src[held] // K]
    recv_w = torch.zeros(src.numel(), dtype=torch.float64, device=src.device)
    recv_w[held] = s["w"].double().reshape(-1)[src[held]]
    return {"rows": rows, "recv_w": recv_w}


def _exact_combine(s):
    src, K = s["lay"]["src"].long(), s["case"]["K"]
    d_y = torch.zeros(s["y"].shape, device=src.device)
    d_w = torch.zeros(s["w"].numel(), dtype=torch.float64, device=src.device)
    held = torch.nonzero(src >= 0).reshape(-1)
    for part in held.split(8192):
        entry = src[part]
        d = s["d_out"][entry // K].double()
        d_y[part] = (s["w"].double().reshape(-1)[entry][:, None] * d).float()
        d_w[entry] = (d * s["y"][part].double()).sum(1)
    return {"d_y": d_y, "d_w": d_w.reshape(s["w"].shape)}
