"""Measured cases of the 4-bit expert weights and of the few-token MoE layer.

Operators (include/moe.h):
  layer       moe_layer_decode      the whole MoE layer for at most 32 tokens, f32 or bf16 expert weights
  layer_w4    moe_layer_decode_w4   the same layer with 4-bit expert weights
  mlp_w4      moe_expert_mlp_w4     the expert MLP on dispatched rows with 4-bit expert weights
  quantize    moe_quantize_w4       expert weights to 4-bit codes with group scales (read back as values)
  dequantize  moe_dequantize_w4     codes and scales to f32 or bf16 weights

4-bit weights: E2M1 codes (sign; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), one power-of-two scale byte s per 32
consecutive k of a row; a code stands for code * 2^(s - 127). Both are laid out in tiles: rows in blocks of 16, k in
blocks of 128 for codes (1024 bytes) and of 512 for scales (256 bytes); see `pack`.
"""
import math

import torch

own = False

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def _layer(name, kind, dtype, T, H, E, k, F, R, C, routing):
    return {"name": name, "kind": kind, "dtype": dtype, "T": T, "H": H, "E": E, "k": k, "F": F, "R": R, "C": C,
            "routing": routing}


def _matrix(name, kind, dtype, L, N, K):
    return {"name": name, "kind": kind, "dtype": dtype, "L": L, "N": N, "K": K}


def listed():
    return [
        # the tiny fp32 layer answering one token: launches and latency are all there is
        _layer("layer f32 tiny, 1 token", "layer", "f32", 1, 128, 8, 2, 256, 1, 1, "uniform"),
        # one user's next token through a Mixtral-8x7B-shaped layer: two experts of 352 MB each
        _layer("layer bf16 mixtral, 1 token", "layer", "bf16", 1, 4096, 8, 2, 14336, 1, 1, "uniform"),
        # a small decode batch through one GPU's share of a Kimi-K2-shaped layer, skewed routing with a capacity
        _layer("layer bf16 kimi, 16 tokens", "layer", "bf16", 16, 7168, 384, 8, 2048, 8, 4, "zipf"),
        # one user's next token through a DeepSeek-V3-shaped share with 4-bit experts
        _layer("layer w4 dsv3, 1 token", "layer_w4", "bf16", 1, 7168, 256, 8, 2048, 8, 1, "uniform"),
        # the largest batch of the few-token layer, 4-bit experts
        _layer("layer w4 kimi, 32 tokens", "layer_w4", "bf16", 32, 7168, 384, 8, 2048, 8, 32, "zipf"),
        # the Kimi-K2-shaped decode workload's expert MLP: few rows per expert, the weights' bytes count
        _layer("mlp w4 kimi decode", "mlp_w4", "bf16", 128, 7168, 384, 8, 2048, 8, 4, "zipf"),
        # the DeepSeek-V3-shaped prefill workload's expert MLP: 1024 rows per local expert, matrix-bound
        _layer("mlp w4 dsv3 prefill", "mlp_w4", "bf16", 4096, 7168, 256, 8, 2048, 8, 128, "uniform"),
        # a short prompt through a small model whose sizes fit no tile
        _layer("mlp w4 ragged", "mlp_w4", "bf16", 301, 1184, 24, 3, 736, 2, 35, "zipf"),
        # making the weights: the gate/up matrices of eight DeepSeek-V3-shaped experts
        _matrix("quantize bf16 8 experts", "quantize", "bf16", 8, 4096, 7168),
        # one small fp32 expert of a ragged model
        _matrix("quantize f32 ragged", "quantize", "f32", 1, 1472, 1184),
        # expanding the down matrices of sixteen such experts
        _matrix("dequantize bf16 16 experts", "dequantize", "bf16", 16, 7168, 2048),
        # three small fp32 ones of the ragged model
        _matrix("dequantize f32 ragged", "dequantize", "f32", 3, 1184, 736),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def _draw_once(rng):
    kind = rng.choice(["layer", "layer", "layer_w4", "layer_w4", "mlp_w4", "mlp_w4", "quantize", "dequantize"])
    if kind in ("quantize", "dequantize"):
        dtype = rng.choice(["f32", "bf16"])
        return {"kind": kind, "dtype": dtype, "L": _log_int(rng, 1, 32), "N": _log_int(rng, 32, 14336, 32),
                "K": _log_int(rng, 32, 14336, 32)}
    step = 8 if kind == "layer" else 32
    R = rng.choice([1, 1, 2, 3, 8])
    E = R * _log_int(rng, 2, 64)
    k = rng.randint(1, min(8, E))
    T = _log_int(rng, 1, 32) if kind != "mlp_w4" else _log_int(rng, 1, 4096)
    C = rng.choice([T, T, max(1, -(-5 * T * k // (4 * E))), max(1, T * k // E)])
    return {"kind": kind, "dtype": rng.choice(["f32", "bf16"]) if kind == "layer" else "bf16", "T": T,
            "H": _log_int(rng, 64, 7168, step), "E": E, "k": k, "F": _log_int(rng, 32, 14336, step), "R": R,
            "C": min(C, T), "routing": rng.choice(["uniform", "zipf"])}


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["kind"], [0, 0])
        t[0], t[1] = max(t[0], w["bytes"]), max(t[1], w["flops"])
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] > top[c["kind"]][0] or w["flops"] > top[c["kind"]][1]:
            continue
        if "E" in c and c["E"] // c["R"] * 3 * c["F"] * c["H"] > 64 * 3 * 2048 * 7168:
            continue  # the weights a state holds
        return c


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def _bias_list(case):
    if case["routing"] == "zipf":
        return [-1.2 * math.log(e + 1.0) for e in range(case["E"])]
    return [0.0] * case["E"]


def _choice_odds(case):
    """The share of tokens that choose each expert: logits are N(b_e, (0.02 sqrt(H))^2), the k largest win."""
    b, sd, k = _bias_list(case), 0.02 * math.sqrt(case["H"]), case["k"]
    lo, hi = min(b) - 12 * sd, max(b) + 12 * sd
    over = lambda cut: [0.5 * math.erfc((cut - v) / (sd * math.sqrt(2.0))) for v in b]
    for _ in range(60):
        mid = 0.5 * (lo + hi)
        lo, hi = (mid, hi) if sum(over(mid)) > k else (lo, mid)
    return over(lo)


def work(case):
    if case["kind"] in ("quantize", "dequantize"):
        n = case["L"] * case["N"] * case["K"]
        wide = n * (4 if case["dtype"] == "f32" else 2)
        packed = n // 2 + n // 32
        # quantize is read back: the packed weights are written and read, the values written
        return {"bytes": 2 * (wide + packed) if case["kind"] == "quantize" else wide + packed, "flops": n}
    T, H, E, k, F, R, C = (case[n] for n in ("T", "H", "E", "k", "F", "R", "C"))
    El = E // R
    odds = _choice_odds(case)
    rows = sum(min(T * p, C) for p in odds)
    # local experts that at least one token's pair reaches
    used = sum(1.0 - math.prod((1.0 - odds[r * El + l]) ** T for r in range(R)) for l in range(El))
    used = min(used, float(T * k))
    esz = 4 if case["dtype"] == "f32" else 2
    wsz = 17.0 / 32.0 if case["kind"].endswith("w4") else esz
    weights = used * 3 * F * H * wsz
    if case["kind"] == "mlp_w4":
        return {"bytes": int(weights + 2 * rows * H * esz), "flops": int(6 * rows * F * H)}
    return {"bytes": int(weights + E * H * 4 + 2 * T * H * esz + T * (E + 2 * k) * 4),
            "flops": int(6 * rows * F * H + 2 * T * E * H)}


# ---------------------------------------------------------------------------------------------------------------------
# 4-bit weights in elementary operations
# ---------------------------------------------------------------------------------------------------------------------

def _encode(w):
    """w [N, K] float32 -> (codes [N, K] uint8 0..15, scale bytes [N, K / 32] uint8)."""
    N, K = w.shape
    g = w.view(N, K // 32, 32)
    m, e = torch.frexp(g.abs().amax(2))           # amax = m 2^e, m in [0.5, 1): amax <= 6 2^E
    E = torch.where(m <= 0.75, e - 3, e - 2)      # 0.75 2^e = 6 2^(e - 3)
    E = torch.where(m == 0, torch.zeros_like(E), E.clamp(-120, 125))
    v = torch.ldexp(g, -E.unsqueeze(2)).abs()
    code = torch.zeros_like(v, dtype=torch.uint8)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (v >= border) if up else (v > border)   # a tie goes to the even code
    code = code | (torch.signbit(g).to(torch.uint8) << 3)
    return code.view(N, K), (E + 127).to(torch.uint8)


def pack(code, scale):
    """Codes [N, K] and scale bytes [N, K / 32] in tiles: codes [N/16, ceil(K/128), 1024], scales
    [N/16, ceil(K/512), 256] (uint8), zero codes and scale byte 127 past K. In a code tile lane
    (n % 16) + 16 ((k % 128) / 32) owns 16 consecutive bytes, 32 k's, the even one in the low nibble; in a scale tile
    the same lane owns 4 bytes, one per 128 k's."""
    N, K = code.shape
    kc, ks = -(-K // 128), -(-K // 512)
    full = torch.zeros(N, kc * 128, dtype=torch.uint8, device=code.device)
    full[:, :K] = code
    full = full[:, 0::2] | (full[:, 1::2] << 4)
    codes = full.view(N // 16, 16, kc, 4, 16).permute(0, 2, 3, 1, 4).reshape(N // 16, kc, 1024).contiguous()
    sc = torch.full((N, ks * 16), 127, dtype=torch.uint8, device=code.device)
    sc[:, :K // 32] = scale
    scales = sc.view(N // 16, 16, ks, 4, 4).permute(0, 2, 4, 1, 3).reshape(N // 16, ks, 256).contiguous()
    return codes, scales


def _decode(codes, scales, K, lut):
    """Packed tiles [N/16, kc, 1024], [N/16, ks, 256] -> float32 [N, K]."""
    nb, kc, ks = codes.shape[0], codes.shape[1], scales.shape[1]
    b = codes.view(nb, kc, 4, 16, 16).permute(0, 3, 1, 2, 4).reshape(nb * 16, kc * 64)
    idx = torch.stack((b & 15, b >> 4), dim=2).view(nb * 16, kc * 128)[:, :K]
    s = scales.view(nb, ks, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(nb * 16, ks * 16)[:, :K // 32]
    v = lut[idx.int()].view(nb * 16, K // 32, 32)
    return torch.ldexp(v, (s.int() - 127).unsqueeze(2)).view(nb * 16, K)


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _weights(case, g, packed):
    """N(0, 0.02^2) expert weights rounded to the activation type; with `packed`, quantised and packed."""
    El, H, F = case["E"] // case["R"], case["H"], case["F"]
    out = []
    for N, K in ((2 * F, H), (H, F)):
        parts = []
        for _ in range(El):
            w = torch.randn(N, K, generator=g, device="cuda").mul_(0.02).to(_dtype(case))
            parts.append(pack(*_encode(w.float())) if packed else w)
        if packed:
            out += [torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])]
        else:
            out.append(torch.stack(parts))
    return out


def _layout(ids, case):
    """The dispatch of given expert ids: kept pairs grouped by expert, by token inside one."""
    T, k, E, C = case["T"], case["k"], case["E"], case["C"]
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    count = torch.bincount(flat, minlength=E)
    first = torch.cumsum(count, 0) - count
    place = torch.empty_like(flat)
    place[order] = torch.arange(T * k, device=flat.device) - first[flat[order]]
    kept = count.clamp(max=C)
    offset = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offset[1:] = torch.cumsum(kept, 0)
    row = torch.where(place < C, offset[flat] + place, torch.full_like(place, -1))
    return {"count": count, "kept": kept, "overflow": count - kept, "offset": offset, "pair_row": row.view(T, k)}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": dict(case), "lut": torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device="cuda")}
    if case["kind"] in ("quantize", "dequantize"):
        L, N, K = case["L"], case["N"], case["K"]
        w = torch.empty(L, N, K, dtype=_dtype(case), device="cuda")
        for l in range(L):
            w[l] = torch.randn(N, K, generator=g, device="cuda").mul_(0.02)
        if case["kind"] == "dequantize":
            parts = [pack(*_encode(w[l].float())) for l in range(L)]
            st["codes"] = torch.stack([p[0] for p in parts])
            st["scales"] = torch.stack([p[1] for p in parts])
        else:
            st["w"] = w
            st["codes"] = torch.empty(L, N // 16, -(-K // 128), 1024, dtype=torch.uint8, device="cuda")
            st["scales"] = torch.empty(L, N // 16, -(-K // 512), 256, dtype=torch.uint8, device="cuda")
        st["values"] = torch.empty(L, N, K, dtype=_dtype(case), device="cuda")
        return st
    T, H, E, k, F, R, C = (case[n] for n in ("T", "H", "E", "k", "F", "R", "C"))
    dt = _dtype(case)
    st["weights"] = _weights(case, g, case["kind"].endswith("w4"))
    bias = torch.tensor(_bias_list(case), device="cuda") if case["routing"] == "zipf" else None
    x = torch.randn(T, H, generator=g, device="cuda").to(dt)
    w_router = torch.randn(E, H, generator=g, device="cuda").mul_(0.02)
    if case["kind"] == "mlp_w4":
        scores = x.double() @ w_router.double().T
        if bias is not None:
            scores += bias.double()
        ids = torch.argsort(scores, dim=1, descending=True, stable=True)[:, :k]
        lay = _layout(ids, case)
        rows_max = min(T * k, E * C)
        send = torch.zeros(rows_max, H, dtype=dt, device="cuda")
        pairs = torch.nonzero(lay["pair_row"].reshape(-1) >= 0).reshape(-1)
        send[lay["pair_row"].reshape(-1)[pairs]] = x[pairs // k]
        st.update(send=send, offset=lay["offset"].tolist(), out=torch.zeros_like(send))
        if own:
            import combine_router_gemm_amd as moe
            layout = moe.Layout(T, k, E, R, C, H, device="cuda")
            layout.expert_count.copy_(lay["count"])
            layout.expert_kept.copy_(lay["kept"])
            layout.expert_overflow.copy_(lay["overflow"])
            layout.expert_offset.copy_(lay["offset"])
            layout.pair_row.copy_(lay["pair_row"])
            layout.row_token[lay["pair_row"].reshape(-1)[pairs]] = (pairs // k).int()
            layout.row_slot[lay["pair_row"].reshape(-1)[pairs]] = (pairs % k).int()
            st["layout"] = layout
            n = moe.moe_expert_mlp_w4_workspace_bytes(T, k, E, R, C, F)
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return st
    st.update(x=x, w_router=w_router, bias=bias, y=torch.empty_like(x),
              logits=torch.empty(T, E, dtype=torch.float32, device="cuda"),
              ids=torch.empty(T, k, dtype=torch.int32, device="cuda"),
              w=torch.empty(T, k, dtype=torch.float32, device="cuda"))
    if own:
        import combine_router_gemm_amd as moe
        n = moe.moe_layer_decode_workspace_bytes(T, H, E, k, F, moe.MOE_F32 if case["dtype"] == "f32" else moe.MOE_BF16)
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _run_own(state, kind)
    if kind == "quantize":
        for l in range(state["case"]["L"]):
            w = state["w"][l].float()
            code, scale = _encode(w)
            v = state["lut"][code.int()].view(w.shape[0], -1, 32)
            state["values"][l] = torch.ldexp(v, (scale.int() - 127).unsqueeze(2)).view_as(w)
        return state["values"]
    if kind == "dequantize":
        for l in range(state["case"]["L"]):
            state["values"][l] = _decode(state["codes"][l], state["scales"][l], state["case"]["K"], state["lut"])
        return state["values"]
    return _plain_mlp(state) if kind == "mlp_w4" else _plain_layer(state)


def _run_own(state, kind):
    import combine_router_gemm_amd as moe
    c = state["case"]
    if kind == "quantize":
        moe.moe_quantize_w4(state["w"], state["codes"], state["scales"])
        moe.moe_dequantize_w4(state["codes"], state["scales"], state["values"])
        return state["values"]
    if kind == "dequantize":
        moe.moe_dequantize_w4(state["codes"], state["scales"], state["values"])
        return state["values"]
    if kind == "mlp_w4":
        moe.moe_expert_mlp_w4(state["send"], state["layout"], *state["weights"], state["out"],
                              workspace=state["workspace"])
        return state["out"]
    call = moe.moe_layer_decode if kind == "layer" else moe.moe_layer_decode_w4
    call(state["x"], state["w_router"], state["bias"], c["k"], c["R"], c["C"], *state["weights"], state["logits"],
         state["ids"], state["w"], state["y"], workspace=state["workspace"])
    return {"y": state["y"], "logits": state["logits"], "ids": state["ids"], "w": state["w"]}


def _plain_mlp(state):
    c = state["case"]
    El, H, F, off = c["E"] // c["R"], c["H"], c["F"], state["offset"]
    gu_c, gu_s, dn_c, dn_s = state["weights"]
    for l in range(El):
        spans = [(off[e], off[e + 1]) for e in range(l, c["E"], El) if off[e + 1] > off[e]]
        if not spans:
            continue
        gu = _decode(gu_c[l], gu_s[l], H, state["lut"])
        dn = _decode(dn_c[l], dn_s[l], F, state["lut"])
        rows = torch.cat([state["send"][a:b] for a, b in spans]).float()
        s = rows @ gu.T
        h = s[:, :F] / (1.0 + torch.exp(-s[:, :F])) * s[:, F:]
        out, at = h @ dn.T, 0
        for a, b in spans:
            state["out"][a:b] = out[at:at + b - a]
            at += b - a
    return state["out"]  # rows past the kept ones stay as they were


def _plain_layer(state):
    c = state["case"]
    T, H, E, k, F, C = (c[n] for n in ("T", "H", "E", "k", "F", "C"))
    El = E // c["R"]
    x = state["x"].float()
    logits = state["x"].double() @ state["w_router"].double().T
    if state["bias"] is not None:
        logits += state["bias"].double()
    ids = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
    s = torch.gather(logits, 1, ids)
    w = torch.exp(s - s[:, :1])
    w = (w / w.sum(1, keepdim=True)).float()
    chosen = torch.zeros(T, E, device="cuda").scatter_(1, ids, 1.0)
    before = torch.cumsum(chosen, 0) - chosen
    kept = torch.gather(before, 1, ids) < C
    le = (ids % El).reshape(-1)
    y = torch.zeros(T, H, device="cuda")
    for p in range(T * k):
        t, l = p // k, le[p:p + 1]
        tiles = [m.index_select(0, l)[0] for m in state["weights"]]
        if c["kind"] == "layer":
            gu, dn = tiles[0].float(), tiles[1].float()
        else:
            gu = _decode(tiles[0], tiles[1], H, state["lut"])
            dn = _decode(tiles[2], tiles[3], F, state["lut"])
        gate_up = gu @ x[t]
        h = gate_up[:F] / (1.0 + torch.exp(-gate_up[:F])) * gate_up[F:]
        y[t] += torch.where(kept[t, p % k], w[t, p % k] * (dn @ h), torch.zeros(H, device="cuda"))
    return {"y": y.to(state["x"].dtype), "logits": logits.float(), "ids": ids.int(), "w": w}


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _exact_values(w):
    """What each element of w [N, K] becomes: the nearest multiple of the step that its magnitude has on the grid."""
    a = w.double().view(w.shape[0], -1, 32)
    top = a.abs().amax(2, keepdim=True)
    E = torch.ceil(torch.log2(top / 6.0))
    E = torch.where(6.0 * torch.exp2(E) < top, E + 1, E)           # log2's own rounding next to a power of two
    E = torch.where(6.0 * torch.exp2(E - 1) >= top, E - 1, E)
    unit = torch.exp2(torch.where(top > 0, E.clamp(-120, 125), torch.zeros_like(E)))
    v = a / unit
    step = torch.where(v.abs() < 2.0, 0.5, torch.where(v.abs() < 4.0, 1.0, 2.0))
    return ((torch.round(v / step) * step).clamp(-6.0, 6.0) * unit).view(w.shape)


def _exact_unpacked(codes, scales, N, K):
    n = torch.arange(N, device="cuda").view(N, 1)
    k = torch.arange(K, device="cuda").view(1, K)
    lane = n % 16 + 16 * (k % 128 // 32)
    kc, ks = codes.shape[1], scales.shape[1]
    byte = codes.reshape(-1)[((n // 16) * kc + k // 128) * 1024 + lane * 16 + k % 32 // 2]
    nib = torch.where(k % 2 == 0, byte & 15, byte >> 4).double()
    s = scales.reshape(-1)[((n // 16) * ks + k // 512) * 256 + lane * 4 + k % 512 // 128].double()
    sign = torch.where(nib >= 8, -1.0, 1.0)
    m = nib % 8
    e = torch.floor(m / 2)
    mag = torch.where(e == 0, m / 2, (1.0 + m % 2 / 2) * torch.exp2(e - 1))
    return sign * mag * torch.exp2(s - 127.0)


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "quantize":
        return torch.stack([_exact_values(st["w"][l]) for l in range(case["L"])])
    if case["kind"] == "dequantize":
        return torch.stack([_exact_unpacked(st["codes"][l], st["scales"][l], case["N"], case["K"])
                            for l in range(case["L"])])
    T, H, E, k, F, R, C = (case[n] for n in ("T", "H", "E", "k", "F", "R", "C"))
    El = E // R

    def expert(l, rows):
        if case["kind"] == "layer":
            gu, dn = st["weights"][0][l].double(), st["weights"][1][l].double()
        else:
            gu = _exact_unpacked(st["weights"][0][l], st["weights"][1][l], 2 * F, H)
            dn = _exact_unpacked(st["weights"][2][l], st["weights"][3][l], H, F)
        g, u = rows @ gu[:F].T, rows @ gu[F:].T
        return (g * torch.sigmoid(g) * u) @ dn.T

    if case["kind"] == "mlp_w4":
        out = torch.zeros(min(T * k, E * C), H, dtype=torch.float64, device="cuda")
        for l in range(El):
            at = [i for e in range(l, E, El) for i in range(st["offset"][e], st["offset"][e + 1])]
            if at:
                out[at] = expert(l, st["send"][at].double())
        return out
    x = st["x"].double()
    logits = torch.stack([(st["w_router"].double() * x[t]).sum(1) for t in range(T)])
    if st["bias"] is not None:
        logits = logits + st["bias"].double()
    host = logits.tolist()
    ids = [sorted(range(E), key=lambda e: (-host[t][e], e))[:k] for t in range(T)]
    picked = torch.stack([logits[t][ids[t]] for t in range(T)])
    w = torch.softmax(picked, dim=1)
    y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for l in sorted({e % El for row in ids for e in row}):
        for e in range(l, E, El):
            who = [t for t in range(T) if e in ids[t]][:C]
            if who:
                y[who] += w[who, [ids[t].index(e) for t in who]].unsqueeze(1) * expert(l, x[who])
    return {"y": y, "logits": logits, "ids": torch.tensor(ids, dtype=torch.int32), "w": w}
