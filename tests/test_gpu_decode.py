"""GPU: the whole layer for a few tokens (moe_layer_decode, moe_layer_decode_w4) against float64 (bounds:
tests/_layer_ref.py), against the four calls, and in the ways a serving loop uses it."""
import pytest
import torch

import combine_router_gemm_amd as moe
import moe_workloads as W
import oracle
from tests._hip_runner import run_layer
from tests._layer_ref import layer, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def inputs(name, T, H, E, k, F, R, dtype, routing, seed):
    cfg = W.small_config(W.workload("tiny-fp32"), seed=seed, name=name, T=T, H=H, E=E, k=k, F=F, R=R,
                         dtype="f32" if dtype == torch.float32 else "bf16", routing=routing)
    return W.make_inputs(cfg, device=DEV)


def pack4(w):
    cs, ss = moe.moe_w4_shapes(*w.shape)
    c, s = torch.empty(cs, dtype=torch.uint8, device=DEV), torch.empty(ss, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_w4(w, c, s)
    v = torch.empty_like(w)
    moe.moe_dequantize_w4(c, s, v)
    return [c, s], v


class Run:
    """Buffers of one layer call; poisoned so that an unwritten output shows."""

    def __init__(self, inp, k, R, C, packs=None, workspace=True):
        x, E = inp["x"], inp["w_router"].shape[0]
        self.inp, self.k, self.R, self.C, self.packs = inp, k, R, C, packs
        T, H = x.shape
        F = inp["w_down"].shape[2]
        self.logits = torch.full((T, E), float("nan"), device=DEV)
        self.ids = torch.full((T, k), -9, dtype=torch.int32, device=DEV)
        self.w = torch.full((T, k), float("nan"), device=DEV)
        self.y = torch.full_like(x, float("nan"))
        n = moe.moe_layer_decode_workspace_bytes(T, H, E, k, F, moe.MOE_BF16 if x.dtype == torch.bfloat16 else moe.MOE_F32)
        self.ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device=DEV) if workspace else None

    def __call__(self, stream=None):
        i = self.inp
        out = (self.logits, self.ids, self.w, self.y)
        if self.packs is None:
            moe.moe_layer_decode(i["x"], i["w_router"], i["bias"], self.k, self.R, self.C, i["w_gate_up"], i["w_down"],
                                 *out, workspace=self.ws, stream=stream)
        else:
            moe.moe_layer_decode_w4(i["x"], i["w_router"], i["bias"], self.k, self.R, self.C, *self.packs, *out,
                                    workspace=self.ws, stream=stream)
        return self

    def outputs(self):
        return [t.clone() for t in (self.logits, self.ids, self.w, self.y)]


def same(a, b):
    return all(torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x,
                           y.view(torch.int16) if y.dtype == torch.bfloat16 else y) for x, y in zip(a, b))


def check(r, gu, dn):
    torch.cuda.synchronize()
    lg = r.logits.cpu()
    ids = r.ids.cpu().long()
    assert torch.equal(ids, torch.from_numpy(oracle.topk_select(lg.numpy(), r.k)).long())
    x = r.inp["x"].cpu()
    bias = None if r.inp["bias"] is None else r.inp["bias"].cpu().double()
    guc, dnc = gu.cpu(), dn.cpu()
    half = 0.0 if x.dtype == torch.float32 else 2.0 ** -16  # h: two bf16 parts
    ref = layer(x.double(), r.inp["w_router"].cpu().double(), bias, r.k, r.R, r.C, ids,
                lambda l: (guc[l].double(), dnc[l].double()), half)
    assert float(((lg.double() - ref["logits"]).abs() / ref["dlogits"].clamp_min(1e-30)).max()) <= 1.0
    assert float(((r.w.cpu().double() - ref["w"]).abs() / ref["dw"]).max()) <= 1.0
    assert within(r.y.cpu(), ref["y"], ref["dy"], x.dtype) <= 1.0


CASES = [
    # name, T, H, E, k, F, R, C, routing
    ("one_token", 1, 128, 8, 2, 256, 1, 1, "uniform"),
    ("one_expert", 3, 64, 1, 1, 32, 1, 3, "uniform"),
    ("k_is_E", 2, 64, 8, 8, 64, 2, 2, "uniform"),
    ("ragged", 5, 168, 60, 3, 104, 3, 5, "zipf"),
    ("tokens_16", 16, 320, 24, 4, 96, 2, 16, "uniform"),
    ("tokens_17", 17, 96, 12, 2, 160, 1, 17, "zipf"),
    ("tokens_32_hot", 32, 256, 16, 2, 64, 1, 32, "hot8"),
    ("capacity", 32, 128, 10, 3, 64, 2, 3, "zipf"),
    ("capacity_zero", 4, 64, 8, 2, 32, 1, 0, "uniform"),
    ("experts_512", 6, 96, 512, 8, 32, 8, 2, "uniform"),
    ("long_k", 2, 2056, 6, 2, 1048, 1, 2, "uniform"),
    ("smallest", 1, 8, 2, 1, 8, 1, 1, "uniform"),
    # H narrow and F long: the down product is split, into more parts than there are steps of chosen experts in the last
    ("split_down", 9, 224, 24, 4, 1504, 2, 9, "uniform"),
    ("split_down_wide_f", 20, 96, 40, 4, 2080, 1, 20, "zipf"),
    ("split_down_few_chosen", 32, 64, 64, 2, 1056, 1, 32, "hot8"),
    # H short and tiles enough: fewer waves share a tile of gate/up
    ("many_tiles", 24, 96, 64, 8, 3104, 1, 24, "uniform"),
    ("many_tiles_hot", 32, 160, 40, 4, 3360, 1, 32, "zipf"),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name,T,H,E,k,F,R,C,routing", CASES, ids=[c[0] for c in CASES])
def test_layer_decode(name, T, H, E, k, F, R, C, routing, dtype):
    print(f"\n[gpu] layer decode {name} {dtype}", flush=True)
    inp = inputs(name, T, H, E, k, F, R, dtype, routing, 800 + T)
    check(Run(inp, k, R, C)(), inp["w_gate_up"], inp["w_down"])


@pytest.mark.parametrize("name,T,H,E,k,F,R,C,routing", [c for c in CASES if c[0] not in ("smallest",)],
                         ids=[c[0] for c in CASES if c[0] not in ("smallest",)])
def test_layer_decode_w4(name, T, H, E, k, F, R, C, routing):
    H, F = -(-H // 32) * 32, -(-F // 32) * 32
    print(f"\n[gpu] layer decode w4 {name}", flush=True)
    inp = inputs(name, T, H, E, k, F, R, torch.bfloat16, routing, 900 + T)
    pg, gu = pack4(inp["w_gate_up"])
    pd, dn = pack4(inp["w_down"])
    check(Run(inp, k, R, C, pg + pd)(), gu, dn)


@pytest.mark.parametrize("T,E,R,C", [(1, 16, 1, 1), (7, 16, 4, 7), (32, 40, 2, 3)])
def test_agrees_with_the_four_calls(T, E, R, C):
    """The same layer through route, dispatch, expert MLP and combine: both are within the stated bf16 tolerance of
    the layer (2e-2 per token), so within twice it of each other; a token that lost every pair is 0 in both."""
    inp = inputs("four", T, 256, E, 4, 192, R, torch.bfloat16, "zipf", 40 + T)
    inp["C"] = C
    four = run_layer(inp, 4, R)
    r = Run(inp, 4, R, C)()
    torch.cuda.synchronize()
    assert torch.equal(r.ids, four["ids"])
    a, b = r.y.double(), four["y"].double()
    zero = b.abs().amax(1) == 0
    assert torch.equal(zero, a.abs().amax(1) == 0)
    assert torch.all((a - b).norm(dim=1) <= 4e-2 * b.norm(dim=1))


def test_ties_and_non_finite_logits_follow_the_router():
    T, H, E, k = 6, 64, 70, 5
    inp = inputs("ties", T, H, E, k, 32, 1, torch.float32, "uniform", 77)
    inp["w_router"].zero_()
    bias = torch.zeros(T, E, device=DEV)
    bias[1, 3], bias[1, 9] = 1.0, 1.0
    bias[2, 4] = float("nan")
    bias[3, :] = float("nan")
    bias[4, 60:] = -0.0
    bias[5, 2], bias[5, 0] = float("inf"), float("-inf")
    inp["bias"] = bias
    r = Run(inp, k, 1, T)()
    torch.cuda.synchronize()
    assert torch.equal(r.ids.cpu().long(), torch.from_numpy(oracle.topk_select(r.logits.cpu().numpy(), k)).long())


@pytest.mark.parametrize("w4", [False, True])
def test_a_bad_token_or_expert_reaches_no_other_token(w4):
    """Token 0 holds a NaN and an infinity; an expert that only token 0 chose has (unpacked) infinite weights."""
    T, H, E, k, F = 4, 64, 8, 2, 32
    inp = inputs("bad", T, H, E, k, F, 1, torch.bfloat16, "uniform", 5)
    bias = torch.zeros(T, E, device=DEV)
    bias[0, 6:] = 100.0
    bias[1:, :4] = 100.0
    inp["bias"] = bias
    inp["w_router"].zero_()
    packs = None
    if w4:
        packs = pack4(inp["w_gate_up"])[0] + pack4(inp["w_down"])[0]
    clean = Run(inp, k, 1, T, packs)().outputs()
    inp["x"][0, 5], inp["x"][0, 9] = float("nan"), float("inf")
    if not w4:
        inp["w_gate_up"][6, 1, 2] = float("inf")
        inp["w_down"][7, 3, 4] = float("nan")
    got = Run(inp, k, 1, T, packs)().outputs()
    assert torch.equal(got[3][1:], clean[3][1:])
    assert not torch.isfinite(got[3][0].float()).all()


@pytest.mark.parametrize("w4", [False, True])
def test_an_infinite_h_stays_infinite(w4):
    """h beyond bf16's range is an infinity, as it is when stored as bf16; its second part must not make it NaN."""
    H = F = 32
    inp = inputs("inf", 1, H, 2, 1, F, 1, torch.bfloat16, "uniform", 8)
    inp["x"].fill_(1.0)
    for n in ("w_gate_up", "w_down"):
        inp[n].zero_()
    inp["w_gate_up"][:, 3, 0] = 2.0 ** 100
    inp["w_gate_up"][:, F + 3, 0] = 2.0 ** 100     # h_3 = 2^200
    inp["w_down"].fill_(1.0)
    packs = pack4(inp["w_gate_up"])[0] + pack4(inp["w_down"])[0] if w4 else None
    y = Run(inp, 1, 1, 1, packs)().y
    assert torch.all(y == float("inf"))


def test_zero_tokens_write_nothing():
    inp = inputs("none", 4, 64, 8, 2, 32, 1, torch.bfloat16, "uniform", 6)
    inp["x"] = inp["x"][:0]
    r = Run(inp, 2, 1, 0)
    r.logits, r.ids, r.w, r.y = r.logits[:0], r.ids[:0], r.w[:0], r.y[:0]
    r()


@pytest.mark.parametrize("w4", [False, True])
def test_streams_workspaces_and_graphs(w4):
    """Eager on two streams at once, a temporary workspace, and two captured graphs replayed in turn with eager work
    between: every result equals the eager one bit for bit."""
    T, H, E, k, F, R = 9, 192, 24, 4, 96, 2
    runs, refs = [], []
    for i in range(2):
        inp = inputs("streams", T, H, E, k, F, R, torch.bfloat16, "zipf", 60 + i)
        packs = pack4(inp["w_gate_up"])[0] + pack4(inp["w_down"])[0] if w4 else None
        runs.append(Run(inp, k, R, T, packs))
        refs.append(runs[i]().outputs())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        runs[0](stream=side)
        runs[1]()
    torch.cuda.synchronize()
    for r, ref in zip(runs, refs):
        assert same(r.outputs(), ref)
        r.ws.fill_(0x5A)
    tmp = Run(runs[0].inp, k, R, T, runs[0].packs, workspace=False)(stream=side)
    junk = torch.full((runs[0].ws.numel(),), 0xA5, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert same(tmp.outputs(), refs[0]) and junk[0] == 0xA5
    graphs = []
    for r in runs:
        with torch.cuda.stream(side):
            r()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r()
        graphs.append(g)
    for rep in range(3):
        for g, r, ref in zip(graphs, runs, refs):
            for t in (r.logits, r.w, r.y):
                t.fill_(-1.0)
            r.ids.fill_(-7)
            g.replay()
            torch.cuda.synchronize()
            assert same(r.outputs(), ref)
            r.ws.fill_(rep)
        assert same(runs[0]().outputs(), refs[0])
        torch.cuda.synchronize()


@pytest.mark.parametrize("w4", [False, True])
def test_weights_past_4_gib(w4):
    # the last experts of 4.5 GiB of gate/up codes, or of 5 GiB of bf16 gate/up weights
    El, H, F, T, k = (330, 7168, 2048, 3, 2) if w4 else (160, 4096, 2048, 3, 2)
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB")
    g = torch.Generator(device=DEV).manual_seed(15)
    cpu = torch.Generator().manual_seed(16)
    x = torch.randn(T, H, generator=cpu).to(torch.bfloat16)
    wr = torch.randn(El, H, generator=cpu) * 0.02
    bias = torch.zeros(El)
    bias[-2:] = 1000.0  # every token chooses the last two
    inp = {"x": x.to(DEV), "w_router": wr.to(DEV), "bias": bias.to(DEV), "w_gate_up": None,
           "w_down": torch.empty(0, H, F)}
    if w4:
        packs = []
        for N, K in ((2 * F, H), (H, F)):
            cs, ss = moe.moe_w4_shapes(El, N, K)
            packs += [torch.randint(0, 256, cs, dtype=torch.uint8, device=DEV, generator=g),
                      torch.randint(118, 122, ss, dtype=torch.uint8, device=DEV, generator=g)]

        def weights(N, K, c, s):
            w = torch.empty(N, K, dtype=torch.bfloat16, device=DEV)
            moe.moe_dequantize_w4(c, s, w)
            return w.cpu()
        gu, dn = {}, {}
        for l in (El - 2, El - 1):
            gu[l], dn[l] = weights(2 * F, H, packs[0][l], packs[1][l]), weights(H, F, packs[2][l], packs[3][l])
    else:
        packs = None
        inp["w_gate_up"] = torch.empty(El, 2 * F, H, dtype=torch.bfloat16, device=DEV).normal_(0, 0.02, generator=g)
        inp["w_down"] = torch.empty(El, H, F, dtype=torch.bfloat16, device=DEV).normal_(0, 0.02, generator=g)
        gu = {l: inp["w_gate_up"][l].cpu() for l in (El - 2, El - 1)}
        dn = {l: inp["w_down"][l].cpu() for l in (El - 2, El - 1)}
    r = Run(inp, k, 1, T, packs)()
    torch.cuda.synchronize()
    ids = r.ids.cpu().long()
    assert sorted(ids[0].tolist()) == [El - 2, El - 1]
    ref = layer(x.double(), wr.double(), bias.double(), k, 1, T, ids, lambda l: (gu[l].double(), dn[l].double()),
                2.0 ** -16)
    assert within(r.y.cpu(), ref["y"], ref["dy"], torch.bfloat16) <= 1.0


@pytest.mark.parametrize("w4", [False, True])
def test_split_layers_in_graphs_that_share_a_workspace(w4):
    """Two layers whose down pass is split, captured with one workspace and replayed one after the other, with the
    workspace overwritten between; more tokens than a tile of gate/up has rows."""
    T, H, E, k, F, R = 24, 96, 40, 4, 2080, 1
    runs, refs, graphs = [], [], []
    side = torch.cuda.Stream()
    for i in range(2):
        inp = inputs("split_graphs", T, H, E, k, F, R, torch.bfloat16, "zipf", 70 + i)
        packs = pack4(inp["w_gate_up"])[0] + pack4(inp["w_down"])[0] if w4 else None
        runs.append(Run(inp, k, R, T, packs))
        runs[i].ws = runs[0].ws
        with torch.cuda.stream(side):
            runs[i]()
        torch.cuda.synchronize()
        refs.append(runs[i].outputs())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            runs[i]()
        graphs.append(g)
    for rep in range(3):
        for r in runs:
            r.y.fill_(-1.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for r, ref in zip(runs, refs):
            assert same(r.outputs(), ref)
        runs[0].ws.fill_(0xFF - rep)
        assert same(runs[1]().outputs(), refs[1])
        torch.cuda.synchronize()
