"""The expert layer and its router on the GPU against plain fp64 implementations."""
import numpy as np
import pytest

import oracle
import synth_inputs
from tests import gpu_util as g
from tests import moe_util as mu

pytestmark = pytest.mark.gpu

FMTS = [f"{w}_{x}" for w in ("nf4", "int4", "fp4", "int4a", "mxfp4") for x in ("f16", "bf16")]


# ---- router

def _route_reference(v, top_k, renorm):
    """ids and weights of one row in fp64 (v: fp64 values as the kernel reads them)."""
    never = np.isnan(v) | (v == -np.inf)
    order = sorted((i for i in range(len(v)) if not never[i]), key=lambda i: (-v[i], i))[:top_k]
    ids, w = np.full(top_k, -1), np.zeros(top_k)
    if order:
        top = v[order[0]]
        ex = np.where(never, 0.0, np.where(v == top, 1.0, np.exp(np.where(np.isinf(v) | never, -np.inf, v) -
                                                                 (top if np.isfinite(top) else 0.0))))
        if np.isinf(top):
            ex = np.where(v == top, 1.0, 0.0)
        total = ex[order].sum() if renorm else ex.sum()
        ids[:len(order)] = order
        w[:len(order)] = ex[order] / total
    return ids, w


def _check_route(logits, top_k, renorm):
    import bit_weight_only_w4_amd as w4

    ids, w = w4.moe_route(logits, top_k, renormalize=renorm)
    v = logits.double().cpu().numpy()
    ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    for t in range(v.shape[0]):
        ri, rw = _route_reference(v[t], top_k, renorm)
        assert np.array_equal(ids[t], ri), t
        # exp within 2 ulp of a rounded difference (|v - top| 2^-24 relative for the differences that
        # matter, below 104), the sum of E terms, one division
        tol = (4 + 104 + v.shape[1]) * 2.0 ** -24 * rw + 2.0 ** -126
        assert np.all(np.abs(w[t] - rw) <= tol), t


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 64, 8), (3, 65, 4), (7, 2, 2), (130, 128, 8),
                                                  (5, 256, 16), (2, 1000, 16), (9, 1024, 1), (33, 16, 16)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(dtype, tokens, experts, top_k, renorm):
    import torch

    gen = torch.Generator().manual_seed(tokens + experts)
    v = (torch.randn(tokens, experts, generator=gen) * 3).to(getattr(torch, dtype)).to(g.device())
    _check_route(v, top_k, renorm)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_ties_masks_and_nonfinite(renorm):
    import torch

    inf, nan = float("inf"), float("nan")
    low = torch.finfo(torch.float32).min
    rows = [[1, 1, 1, 1, 1, 1], [0.0, -0.0, 0.0, -0.0, -1, -1], [-inf, -inf, 2, -inf, -inf, -inf],
            [-inf] * 6, [nan] * 6, [nan, 3, nan, 3, -inf, 2], [low] * 6, [low, 0, low, low, 0, low],
            [inf, 0, inf, 5, -inf, nan], [1e38, -1e38, 1e38, 0, 1, 2], [-5, -4, -3, -2, -1, -0.5],
            [1e-45, 0, -1e-45, 0, 0, 0]]
    v = torch.tensor(rows, dtype=torch.float32, device=g.device())
    for k in (1, 3, 6):
        _check_route(v, k, renorm)


def test_route_outputs_given_streams_and_repeats():
    import torch

    import bit_weight_only_w4_amd as w4

    v = torch.randn(50, 40, device=g.device())
    a = w4.moe_route(v, 5)
    ids = torch.full((50, 5), 7, dtype=torch.int32, device=g.device())
    w = torch.full((50, 5), 7.0, device=g.device())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = w4.moe_route(v, 5, ids=ids, weights=w, stream=s)
    torch.cuda.synchronize()
    assert b[0] is ids and b[1] is w
    assert torch.equal(a[0], ids) and torch.equal(a[1], w)


# ---- layer

def _run(c, **kw):
    import bit_weight_only_w4_amd as w4

    return w4.moe(*mu.to_device(c, g.device()), **kw)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", [
    (1, 128, 128, 4, 2), (1, 256, 128, 1, 1), (2, 640, 384, 6, 3), (5, 384, 640, 3, 2), (17, 128, 256, 5, 4),
    (40, 256, 128, 2, 2), (33, 128, 128, 40, 2)])
def test_layer(fmt, tokens, hidden, inter, experts, top_k):
    c = mu.case(fmt, tokens, hidden, inter, experts, top_k, seed=tokens + hidden + inter)
    mu.check(_run(c), c)


@pytest.mark.parametrize("fmt", ["nf4_f16", "fp4_bf16", "mxfp4_f16"])
@pytest.mark.parametrize("tokens,hidden,inter", [(1, 64, 64), (3, 192, 320), (8, 1088, 64), (6, 64, 1088)])
def test_layer_sizes_of_64(fmt, tokens, hidden, inter):
    c = mu.case(fmt, tokens, hidden, inter, 5, 2, seed=hidden + inter)
    mu.check(_run(c), c)


@pytest.mark.parametrize("fmt", ["int4_bf16", "mxfp4_bf16", "nf4_f16"])
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 6, 9, 16, 31, 64, 100])
def test_layer_token_counts(fmt, tokens):
    c = mu.case(fmt, tokens, 256, 256, 8, 3, seed=tokens)
    mu.check(_run(c), c)


@pytest.mark.parametrize("fmt", ["int4a_f16", "mxfp4_bf16"])
def test_every_token_on_one_expert_and_slots_of_one_expert(fmt):
    """All pairs in one expert (more than one chunk of columns), and an expert in several slots."""
    for tokens in (1, 7, 50):
        c = mu.case(fmt, tokens, 256, 128, 12, 4, seed=3)
        c["ids"][:] = 7
        mu.check(_run(c), c)
        c["ids"][:, 2:] = 11
        mu.check(_run(c), c)


@pytest.mark.parametrize("fmt", ["nf4_bf16", "int4_f16"])
@pytest.mark.parametrize("tokens", [1, 4, 30])
def test_absent_slots(fmt, tokens):
    """Ids outside [0, E) add nothing, whatever their weights; a token without experts gets zeros."""
    import torch

    c = mu.case(fmt, tokens, 128, 128, 6, 4, seed=tokens)
    rng = np.random.default_rng(tokens)
    gone = rng.random(c["ids"].shape) < 0.5
    c["ids"][gone] = rng.choice([-1, 6, -2 ** 31, 2 ** 31 - 1], size=int(gone.sum()))
    c["ids"][0] = -1
    clean = c["weights"].copy()
    c["weights"][(c["ids"] < 0) | (c["ids"] >= 6)] = np.nan
    y = _run(c, y=torch.full((tokens, 128), float("nan"), device=g.device()))
    assert torch.equal(y[0], torch.zeros_like(y[0]))
    c["weights"] = clean
    mu.check(y, c)


def test_absent_everywhere():
    import torch

    c = mu.case("mxfp4_bf16", 9, 128, 64, 6, 2, seed=1)
    c["ids"][:] = -1
    y = _run(c, y=torch.full((9, 128), float("nan"), device=g.device()))
    assert torch.equal(y, torch.zeros_like(y))


@pytest.mark.parametrize("fmt", ["fp4_bf16", "int4_f16"])
@pytest.mark.parametrize("tokens", [3, 40])
def test_nonfinite_tokens_stay_alone(fmt, tokens):
    import torch

    c = mu.case(fmt, tokens, 256, 128, 3, 2, seed=5)
    args = list(mu.to_device(c, g.device()))
    args[0] = args[0].clone()
    args[0][1, 3], args[0][2, 200] = float("inf"), float("nan")
    import bit_weight_only_w4_amd as w4

    y = w4.moe(*args)
    assert not torch.isfinite(y[1]).any() and torch.isnan(y[2]).all()
    mu.check(y, c, rows=[t for t in range(tokens) if t not in (1, 2)])


@pytest.mark.parametrize("fmt", ["int4_f16", "fp4_f16", "mxfp4_bf16"])
def test_large_products_between_the_matrices(fmt):
    """h beyond fp16's range: the planes between the products keep fp32's."""
    c = mu.case(fmt, 3, 128, 128, 2, 2, seed=2, sigma=30.0)
    y = _run(c)
    assert float(y.abs().max()) > 65504
    mu.check(y, c)


def test_large_experts_and_repeats():
    """A shape with several quads per K group; the same call gives the same bits."""
    import torch

    c = mu.case("nf4_bf16", 3, 2176, 1088, 3, 2, seed=9)
    args = mu.to_device(c, g.device())
    import bit_weight_only_w4_amd as w4

    y = w4.moe(*args)
    mu.check(y, c)
    for _ in range(3):
        assert torch.equal(w4.moe(*args), y)


def test_workspace_streams_and_capture():
    """A given workspace, another stream, and replays of a captured router and layer with new inputs
    in the captured buffers, each replay against the eager result."""
    import torch

    import bit_weight_only_w4_amd as w4

    dev = g.device()
    fmt, tokens, hidden, inter, experts, top_k = "mxfp4_bf16", 6, 256, 192, 16, 4
    c = mu.case(fmt, tokens, hidden, inter, experts, top_k, seed=4)
    args = list(mu.to_device(c, dev))
    ws = torch.full((w4.moe_workspace_bytes(fmt, tokens, hidden, inter, experts, top_k),), 255,
                    dtype=torch.uint8, device=dev)
    y = w4.moe(*args, workspace=ws)
    mu.check(y, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2 = w4.moe(*args, stream=s)
    s.synchronize()
    assert torch.equal(y, y2)

    logits = torch.randn(tokens, experts, device=dev)
    out = torch.empty(tokens, hidden, device=dev)
    args[1], args[2] = w4.moe_route(logits, top_k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.moe_route(logits, top_k, ids=args[1], weights=args[2])
        w4.moe(*args, y=out, workspace=ws)
    for i in range(4):
        logits.copy_(torch.randn(tokens, experts, device=dev))
        args[0].copy_(torch.randn(tokens, hidden, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        ids, w = w4.moe_route(logits, top_k)
        eager = w4.moe(args[0], ids, w, *args[3:])
        assert torch.equal(eager, out), i


def test_router_and_layer_together_match_the_plain_layer():
    """Quantize, route and run a layer with the library alone, against the fp64 layer."""
    import torch

    import bit_weight_only_w4_amd as w4

    dev = g.device()
    fmt, tokens, hidden, inter, experts, top_k = "mxfp4_f16", 12, 256, 128, 10, 3
    c = mu.case(fmt, tokens, hidden, inter, experts, top_k, seed=8)
    router = torch.from_numpy(synth_inputs.weights(experts, hidden, sigma=0.1, seed=1)).to(dev)
    x = mu.to_device(c, dev)[0]
    gu = synth_inputs.weights(experts * 2 * inter, hidden, sigma=0.05, seed=8)
    dn = synth_inputs.weights(experts * hidden, inter, sigma=0.05, seed=9)
    gp, gs = w4.quantize(fmt, g.to_dev_f32(gu))
    dp, ds = w4.quantize(fmt, g.to_dev_f32(dn))
    ids, w = w4.moe_route(x.float() @ router.t(), top_k)
    y = w4.moe(x, ids, w, gp.view(experts, 2 * inter, -1), gs.view(experts, 2 * inter, -1),
               dp.view(experts, hidden, -1), ds.view(experts, hidden, -1), fmt)
    c["ids"], c["weights"] = ids.cpu().numpy(), w.cpu().numpy()
    mu.check(y, c)


# ---- every way of launching the products: a wave per pair, shared products with K groups, many tokens

LAUNCHES = [(7, 128, 128, 8, 1), (4, 128, 192, 8, 2), (3, 192, 128, 7, 2),    # around as many pairs as experts
            (16, 320, 128, 3, 1), (9, 128, 320, 4, 3),                         # K groups, up to 8 pairs an expert
            (20, 384, 256, 4, 2), (96, 128, 128, 192, 6), (130, 256, 192, 3, 2)]  # many tokens


@pytest.mark.parametrize("fmt", ["nf4_bf16", "int4_f16", "fp4_bf16", "int4a_bf16", "mxfp4_f16"])
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", LAUNCHES)
def test_launches(fmt, tokens, hidden, inter, experts, top_k):
    if fmt.startswith("int4"):
        hidden, inter = (hidden + 127) // 128 * 128, (inter + 127) // 128 * 128
    c = mu.case(fmt, tokens, hidden, inter, experts, top_k, seed=tokens + experts)
    mu.check(_run(c), c)


@pytest.mark.parametrize("fmt", ["nf4_f16", "int4_bf16", "int4a_f16", "mxfp4_bf16", "fp4_f16"])
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", [
    (1, 16768, 128, 2, 2),   # a wave's window of the up product more than once
    (1, 128, 1664, 6, 5),    # and of the down product
    (16, 4224, 128, 4, 1), (16, 128, 4224, 4, 1),   # windows that waves share
    (5, 4224, 2432, 2, 1),
    (40, 2432, 4224, 2, 1), (70, 4224, 640, 1, 1)])  # scale windows, odd numbers of quads
def test_long_rows(fmt, tokens, hidden, inter, experts, top_k):
    c = mu.case(fmt, tokens, hidden, inter, experts, top_k, seed=tokens + hidden)
    mu.check(_run(c), c)


@pytest.mark.parametrize("tokens,experts,top_k", [(2, 40, 16), (1, 1, 16), (9, 1, 1), (3, 1024, 2), (300, 1024, 4),
                                                  (900, 1024, 4)])
def test_most_slots_and_experts(tokens, experts, top_k):
    c = mu.case("mxfp4_bf16", tokens, 64, 64, experts, top_k, seed=experts + tokens)
    mu.check(_run(c), c)


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 4, 2), (8, 4, 2), (40, 4, 2)])
def test_nan_scale_bytes_reach_their_rows_alone(tokens, experts, top_k):
    """A scale byte of 255 in a down row makes that output NaN for the tokens of its expert; in a gate or up row
    it makes that h NaN, and with it every output of its expert's tokens."""
    import torch

    import bit_weight_only_w4_amd as w4

    c = mu.case("mxfp4_bf16", tokens, 320, 192, experts, top_k, seed=6)
    has = (c["ids"] == 2).any(1)
    if not has.any():
        c["ids"][0, 0], has[0] = 2, True
    args = list(mu.to_device(c, g.device()))
    clean = w4.moe(*args)
    scales = args[6].clone()
    scales[2, 77, 5] = 255
    y = w4.moe(*args[:6], scales, args[7])
    want = torch.zeros_like(y, dtype=torch.bool)
    want[torch.from_numpy(has).to(y.device), 77] = True
    assert torch.equal(torch.isnan(y), want) and torch.equal(y[~want], clean[~want])
    for row in (33, 192 + 60):
        scales = args[4].clone()
        scales[2, row, 9] = 255
        y = w4.moe(*args[:4], scales, *args[5:])
        want = torch.from_numpy(has).to(y.device)
        assert torch.isnan(y[want]).all() and torch.equal(y[~want], clean[~want])


@pytest.mark.parametrize("tokens", [2, 12, 60])
def test_operands_off_by_one_element(tokens):
    """ids, weights, scales and y need 4-byte alignment alone; what lies around y stays."""
    import torch

    import bit_weight_only_w4_amd as w4

    for fmt in ("mxfp4_f16", "nf4_bf16"):
        c = mu.case(fmt, tokens, 192, 128, 6, 2, seed=7)
        args = list(mu.to_device(c, g.device()))

        def shifted(t):
            n = 4 // t.element_size()
            buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
            buf[n:] = t.reshape(-1)
            return buf[n:].view(t.shape)

        want = w4.moe(*args)
        for i in (1, 2, 4, 6):
            args[i] = shifted(args[i])
        buf = torch.full((tokens * 192 + 2,), 3.0, device=g.device())
        w4.moe(*args, y=buf[1:-1].view(tokens, 192))
        assert torch.equal(buf[1:-1].view(tokens, 192), want)
        assert float(buf[0]) == 3.0 and float(buf[-1]) == 3.0


@pytest.mark.parametrize("tokens", [4, 60])
def test_two_streams_at_once(tokens):
    import torch

    import bit_weight_only_w4_amd as w4

    cases = [mu.case("int4_bf16", tokens, 256, 256, 6, 2, seed=s) for s in (1, 2)]
    args = [mu.to_device(c, g.device()) for c in cases]
    want = [w4.moe(*a) for a in args]
    size = w4.moe_workspace_bytes("int4_bf16", tokens, 256, 256, 6, 2)
    ws = [torch.empty(size, dtype=torch.uint8, device=g.device()) for _ in args]
    ys = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, y, b, s in zip(args, ys, ws, streams):
            w4.moe(*a, y=y, workspace=b, stream=s)
    torch.cuda.synchronize()
    for y, w in zip(ys, want):
        assert torch.equal(y, w)


@pytest.mark.parametrize("fmt", ["int4a_f16", "mxfp4_bf16"])
def test_capture_of_many_tokens(fmt):
    """The sorted pairs are made anew by every replay."""
    import torch

    import bit_weight_only_w4_amd as w4

    dev = g.device()
    tokens, hidden, inter, experts, top_k = 70, 256, 128, 5, 2
    c = mu.case(fmt, tokens, hidden, inter, experts, top_k, seed=4)
    args = list(mu.to_device(c, dev))
    out = torch.empty(tokens, hidden, device=dev)
    ws = torch.empty(w4.moe_workspace_bytes(fmt, tokens, hidden, inter, experts, top_k), dtype=torch.uint8, device=dev)
    w4.moe(*args, y=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.moe(*args, y=out, workspace=ws)
    rng = np.random.default_rng(3)
    for i in range(4):
        c["ids"] = rng.integers(-1, experts + 1 if i % 2 else 2, size=(tokens, top_k)).astype(np.int32)
        args[1].copy_(torch.from_numpy(c["ids"]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(w4.moe(*args), out), i
        mu.check(out, c)


def test_experts_past_4_gib():
    """The last expert of weights that pass 32-bit offsets."""
    import torch

    import bit_weight_only_w4_amd as w4

    dev = g.device()
    experts, hidden, inter = 1024, 2304, 2048
    gen = torch.Generator(device=dev).manual_seed(1)

    def matrix(n, k):
        p = torch.randint(0, 256, (experts, n, k // 2), dtype=torch.uint8, device=dev, generator=gen)
        s = torch.randint(0x3C00, 0x3C80, (experts, n, k // 128), dtype=torch.int16, device=dev, generator=gen)
        return p, s

    gu, dn = matrix(2 * inter, hidden), matrix(hidden, inter)
    assert gu[0].numel() > 2 ** 32
    last = []
    for p, sc in (gu, dn):
        p, sc = p[-1].cpu().numpy(), sc[-1].cpu().numpy().view(np.uint16)
        hat = oracle.dequant("int4", p, sc)
        mag = hat + 48 * np.repeat(oracle.bf16_bits_to_f64(sc), 128, axis=1)
        last.append((None, None, hat[None], mag[None]))
    for tokens in (1, 3500):
        x = (torch.randn(tokens, hidden, device=dev, generator=gen) / 16).half()
        ids = torch.full((tokens, 1), experts - 1, dtype=torch.int32, device=dev)
        weights = torch.rand(tokens, 1, device=dev, generator=gen)
        y = w4.moe(x, ids, weights, *gu, *dn, "int4_f16")
        rows = [0, tokens // 2, tokens - 1]
        mu.check(y[rows], dict(fmt="int4_f16", x=x[rows].cpu().numpy().view(np.uint16), ids=np.zeros((3, 1), np.int32),
                               weights=weights[rows].cpu().numpy(), gu=last[0], dn=last[1]))


def test_refusals_of_device_tensors():
    import torch

    import bit_weight_only_w4_amd as w4

    args = list(mu.to_device(mu.case("fp4_f16", 4, 128, 64, 4, 2, seed=1), g.device()))
    wrong = {0: [args[0].t().contiguous().t(), args[0].bfloat16(), args[0][:3], args[0][:, :64].contiguous()],
             1: [args[1].long(), args[1].t().contiguous().t(), args[1][:2]],
             2: [args[2].half(), args[2][:, :1]],
             3: [args[3][:, :64], args[3].view(torch.int8), args[3][0]],
             4: [args[4][:, :, :1], args[4].double()],
             5: [args[5][:3], args[5].transpose(1, 2)],
             6: [args[6][:3]]}
    for i, bad in wrong.items():
        for b in bad:
            with pytest.raises((ValueError, TypeError, w4.W4Error)):
                w4.moe(*args[:i], b, *args[i + 1:])
    for y in (torch.empty(4, 64, device=g.device()), torch.empty(4, 128, device=g.device()).half(),
              torch.empty(4, 128)):
        with pytest.raises((ValueError, TypeError, w4.W4Error)):
            w4.moe(*args, y=y)
    with pytest.raises((ValueError, TypeError, w4.W4Error)):
        w4.moe(*args, workspace=torch.empty(64, dtype=torch.uint8, device=g.device()))
    with pytest.raises((ValueError, TypeError, w4.W4Error)):
        w4.moe(*args, y=args[0].view(torch.float32))  # x itself: too small, and the wrong shape
    big = torch.zeros(4 * 128 * 4 + 4 * 128 * 2, dtype=torch.uint8, device=g.device())
    x = big[:4 * 128 * 2].view(torch.float16).view(4, 128)
    y = big[512:512 + 4 * 128 * 4].view(torch.float32).view(4, 128)
    with pytest.raises((ValueError, TypeError, w4.W4Error)):
        w4.moe(x, *args[1:], y=y)  # y over x
