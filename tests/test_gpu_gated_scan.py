"""GPU checks of the per-channel gated scan, its gradients and its decode step
against the recurrence in 64 bits.

Tolerances. The kernels work in fp32: a step's decay and input carry a relative
error of at most 2^-21 (exp2 2^-22, softplus 2^-22, the products), and every
output is a sum of products of at most 2 L + 32 such factors, so with M the same
formula evaluated on absolute values (which bounds every partial sum),

    |got - ref| <= (2 L + 32) 2^-21 M + r |ref|

with r = 2^-8 for bf16 outputs (one rounding, half an ulp is 2^-9, and the ulp
of a value next to a power of two) and 2^-23 for fp32 ones.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_ssd_chunked_gb300 import build
    build.build()


def make(b, L, d, io, seed, packed=False, with_D=True, with_init=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    dt0 = torch.exp(torch.rand(d, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    t = {
        "x": n(b, L, d).to(io), "dt": n(b, L, d).to(io), "dt_bias": dt0 + torch.log(-torch.expm1(-dt0)),
        "A": -torch.exp(torch.rand(d, generator=g, device="cuda") * math.log(16.0)),
        "D": n(d) if with_D else None, "init": n(b, d) if with_init else None,
        "dy": n(b, L, d).to(io), "dfin": n(b, d), "seq": None,
    }
    if packed:
        cuts = torch.rand(b, L, generator=g, device="cuda") < 0.08
        t["seq"] = torch.cumsum(cuts.int(), 1, dtype=torch.int32)
    return t


def reference(t, absolute=False):
    """Forward and gradients in 64 bits, token by token; with `absolute`, on absolute values."""
    f = (lambda v: None if v is None else v.double().abs()) if absolute else \
        (lambda v: None if v is None else v.double())
    x, dy, dfin = f(t["x"]), f(t["dy"]), f(t["dfin"])
    v = t["dt"].double() + t["dt_bias"].double()
    delta = torch.logaddexp(v, torch.zeros_like(v))
    a = torch.exp(delta * t["A"].double())
    A = t["A"].double().abs() if absolute else t["A"].double()
    b, L, d = x.shape
    zero = torch.zeros(b, d, dtype=torch.float64, device=x.device)
    D = zero[0] if t["D"] is None else f(t["D"])
    init = zero if t["init"] is None else f(t["init"])
    if t["seq"] is not None:
        a[:, 1:][t["seq"][:, 1:] != t["seq"][:, :-1]] = 0
    h, hs = init, [init]
    for i in range(L):
        h = a[:, i] * h + delta[:, i] * x[:, i]
        hs.append(h)
    hs = torch.stack(hs, 1)
    g, carry = torch.empty_like(x), dfin
    for i in range(L - 1, -1, -1):
        g[:, i] = dy[:, i] + carry
        carry = a[:, i] * g[:, i]
    dlog = a * g * hs[:, :-1]
    ddt = (g * x + A * dlog) * torch.sigmoid(v)
    return {"y": hs[:, 1:] + D * x, "final_state": h, "dx": delta * g + D * dy, "ddt": ddt, "ddt_bias": ddt.sum((0, 1)),
            "dA": (dlog * delta).sum((0, 1)), "dD": (dy * x).sum((0, 1)), "dinit_state": carry}


def run(t, **kw):
    import mamba_ssd_chunked_gb300 as pkg
    y, fin, ch = pkg.ssd_gated_scan(t["x"], t["dt"], t["dt_bias"], t["A"], t["D"], init_state=t["init"],
                                    seq_idx=t["seq"], return_chunk_states=True, **kw)
    g = pkg.ssd_gated_scan_bwd(t["dy"], t["x"], t["dt"], t["dt_bias"], t["A"], ch, D=t["D"], seq_idx=t["seq"],
                               dfinal_state=t["dfin"], **kw)
    out = dict(zip(("y", "final_state", "dx", "ddt", "ddt_bias", "dA", "dD", "dinit_state"), (y, fin, *g)))
    torch.cuda.synchronize()
    assert pkg.ssd_device_status() == 0
    return out


def check(got, t, what=""):
    ref, most = reference(t), reference(t, absolute=True)
    L = t["x"].shape[1]
    for k, v in got.items():
        if v is None:
            continue
        r = 2.0 ** -8 if v.dtype == torch.bfloat16 else 2.0 ** -23
        bound = (2 * L + 32) * 2.0 ** -21 * most[k] + r * ref[k].abs()
        off = ((v.double() - ref[k]).abs() - bound).max().item()
        assert off <= 0, f"{what} {k}: {off:.3e} over the bound"


DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# (b, L, d): one token, the ends of a thread's run and of a tile, one tile and a
# token, several groups of tiles, odd channel counts, channels past a warp's width
SHAPES = [(1, 1, 64), (3, 1, 1), (2, 7, 33), (1, 8, 130), (2, 63, 65), (1, 64, 64), (2, 65, 70), (1, 200, 257),
          (2, 2048, 66), (1, 2049, 3), (1, 4230, 40), (3, 1021, 771)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_the_recurrence(shape, io):
    t = make(*shape, DTYPES[io], seed=sum(shape))
    check(run(t), t, f"{shape} {io}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 300, 70), (1, 2500, 33), (3, 65, 64)])
def test_packed_sequences(shape, io):
    t = make(*shape, DTYPES[io], seed=7, packed=True)
    check(run(t), t, f"{shape} {io}")


def test_every_token_its_own_sequence():
    t = make(2, 130, 34, torch.float32, seed=8)
    t["seq"] = torch.arange(130, device="cuda", dtype=torch.int32).repeat(2, 1).contiguous()
    got = run(t)
    check(got, t)
    x, v = t["x"].double(), t["dt"].double() + t["dt_bias"].double()
    alone = torch.logaddexp(v, torch.zeros_like(v)) * x + t["D"].double() * x
    assert ((got["y"].double() - alone)[:, 1:].abs() <= 1e-5 * (1 + alone[:, 1:].abs())).all()


@pytest.mark.parametrize("with_D,with_init", [(False, True), (True, False), (False, False)])
def test_absent_inputs(with_D, with_init):
    t = make(2, 150, 40, torch.float32, seed=9, with_D=with_D, with_init=with_init)
    t["dfin"] = torch.zeros_like(t["dfin"])
    got = run(t)
    assert (got["dD"] is None) == (not with_D)
    check(got, t)
    import mamba_ssd_chunked_gb300 as pkg
    _, _, ch = pkg.ssd_gated_scan(t["x"], t["dt"], t["dt_bias"], t["A"], t["D"], init_state=t["init"],
                                  return_chunk_states=True)
    g = pkg.ssd_gated_scan_bwd(t["dy"], t["x"], t["dt"], t["dt_bias"], t["A"], ch, D=t["D"])  # no dfinal_state
    for k, v in zip(("dx", "ddt", "ddt_bias", "dA", "dD", "dinit_state"), g):
        assert v is None or torch.equal(v, got[k])


@pytest.mark.parametrize("offset", [0, 1, 2])
def test_slices_of_a_projection(offset):
    """x, dt and dy inside wider rows, at offsets that do and do not fit two-element accesses."""
    b, L, d = 2, 150, 64
    t = make(b, L, d, torch.bfloat16, seed=10)
    want = run(t)
    wide = torch.zeros(b, L, 3 * d + 6, dtype=torch.bfloat16, device="cuda")
    s = dict(t)
    for i, k in enumerate(("x", "dt", "dy")):
        wide[..., offset + i * d:offset + (i + 1) * d] = t[k]
        s[k] = wide[..., offset + i * d:offset + (i + 1) * d]
    got = run(s)
    for k in want:
        assert torch.equal(want[k], got[k]), k
    import mamba_ssd_chunked_gb300 as pkg
    _, _, ch = pkg.ssd_gated_scan(t["x"], t["dt"], t["dt_bias"], t["A"], t["D"], init_state=t["init"],
                                  return_chunk_states=True)
    grad = torch.full((b, L, 2 * d + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, ddt = grad[..., offset:offset + d], grad[..., offset + d + 1:offset + 2 * d + 1]
    pkg.ssd_gated_scan_bwd(t["dy"], t["x"], t["dt"], t["dt_bias"], t["A"], ch, D=t["D"], dfinal_state=t["dfin"], dx=dx,
                           ddt=ddt)
    assert torch.equal(dx, want["dx"]) and torch.equal(ddt, want["ddt"])
    used = torch.zeros(2 * d + 5, dtype=torch.bool)
    used[offset:offset + d] = True
    used[offset + d + 1:offset + 2 * d + 1] = True
    assert (grad[..., ~used.cuda()] == 7.0).all(), "nothing outside the slices is written"


def test_runs_repeat_bit_for_bit():
    t = make(2, 5000, 200, torch.bfloat16, seed=11)
    first = run(t)
    for _ in range(3):
        again = run(t)
        for k in first:
            assert torch.equal(first[k], again[k]), k


def test_another_stream():
    t = make(2, 700, 96, torch.bfloat16, seed=12)
    want = run(t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(t, stream=s.cuda_stream)
    with torch.cuda.stream(s):
        inside = run(t)
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(want[k], got[k]) and torch.equal(want[k], inside[k]), k


def test_graph_replay():
    import mamba_ssd_chunked_gb300 as pkg
    t = make(1, 3000, 64, torch.float32, seed=13)
    want = run(t)["y"]
    pkg.ssd_gated_scan(t["x"], t["dt"], t["dt_bias"], t["A"], t["D"], init_state=t["init"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, fin, _ = pkg.ssd_gated_scan(t["x"], t["dt"], t["dt_bias"], t["A"], t["D"], init_state=t["init"])
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [63, 64, 129])
def test_rows_that_start_anywhere(d, io):
    """Each input with its own row stride and first element, odd and even, next to values that must not matter;
    some begin or end where their allocation does."""
    b, L = 2, 700
    t = make(b, L, d, DTYPES[io], seed=15, packed=True)
    want = run(t)
    for starts in ((0, 1, 2), (1, 0, 1), (3, 2, 0)):
        s = dict(t)
        for k, extra, start in zip(("x", "dt", "dy"), (3, 2, 5), starts):
            wide = torch.full((b, L, d + extra), float("nan"), dtype=DTYPES[io], device="cuda")
            start = min(start, extra)
            wide[..., start:start + d] = t[k]
            s[k] = wide[..., start:start + d]
        got = run(s)
        for k in want:
            assert torch.equal(want[k], got[k]), (starts, k)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 77])
def test_decode_steps_reproduce_the_scan(io, d):
    import mamba_ssd_chunked_gb300 as pkg
    b, L = 3, 21
    t = make(b, L, d, DTYPES[io], seed=14)
    ref, most = reference(t), reference(t, absolute=True)
    state = t["init"].clone()
    r = 2.0 ** -8 if io == "bf16" else 2.0 ** -23
    for i in range(L):
        y = pkg.ssd_gated_scan_step(t["x"][:, i], t["dt"][:, i], t["dt_bias"], t["A"], t["D"], state=state)
        bound = (2 * L + 32) * 2.0 ** -21 * most["y"][:, i] + r * ref["y"][:, i].abs()
        assert ((y.double() - ref["y"][:, i]).abs() <= bound).all()
    assert ((state.double() - ref["final_state"]).abs() <= (2 * L + 32) * 2.0 ** -21 * most["final_state"]).all()


@pytest.mark.parametrize("d", [4096, 4097])
def test_offsets_past_32_bits(d):
    """More than 2^31 elements: the first and the last sequence's first and last tokens against their own scans."""
    import mamba_ssd_chunked_gb300 as pkg
    b, L, n = 2, 270000, 240
    t = make(1, n, d, torch.bfloat16, seed=16)
    g = torch.Generator(device="cuda").manual_seed(17)
    for k in ("x", "dt", "dy"):
        t[k] = torch.randn(b, L, d, generator=g, device="cuda", dtype=torch.bfloat16)
    t["init"] = torch.randn(b, d, generator=g, device="cuda")
    t["dfin"] = torch.randn(b, d, generator=g, device="cuda")
    y, fin, ch = pkg.ssd_gated_scan(t["x"], t["dt"], t["dt_bias"], t["A"], t["D"], init_state=t["init"],
                                    return_chunk_states=True)
    got = pkg.ssd_gated_scan_bwd(t["dy"], t["x"], t["dt"], t["dt_bias"], t["A"], ch, D=t["D"], dfinal_state=t["dfin"])
    torch.cuda.synchronize()
    assert pkg.ssd_device_status() == 0
    chunk = -(-L // ch.shape[1])
    for i in range(b):
        first = {**t, **{k: t[k][i:i + 1, :n] for k in ("x", "dt", "dy")}, "init": t["init"][i:i + 1],
                 "dfin": torch.zeros(1, d, device="cuda")}
        check({"y": y[i:i + 1, :n]}, first, f"first tokens of {i}")
        at = (L - n) // chunk * chunk  # a saved state, at least n tokens before the end
        last = {**t, **{k: t[k][i:i + 1, at:] for k in ("x", "dt", "dy")}, "init": ch[i:i + 1, at // chunk],
                "dfin": t["dfin"][i:i + 1]}
        check({"y": y[i:i + 1, at:], "final_state": fin[i:i + 1], "dx": got[0][i:i + 1, at:], "ddt": got[1][i:i + 1, at:]},
              last, f"last tokens of {i}")


def test_extreme_gates():
    """Gates that saturate both ways, and a decay that vanishes: no NaN, and the exact limits."""
    t = make(1, 130, 8, torch.float32, seed=15)
    t["dt"][:, :, 0] = 200.0     # delta = 200, a = 0: h = delta x
    t["dt"][:, :, 1] = -200.0    # delta = 0 (below fp32's range), a = 1: h = init
    t["dt"][:, 64, 2] = math.inf  # one infinite gate: a = 0, h = inf x from there on
    t["dt"][:, :, 3] = -math.inf
    t["x"][:, 64, 2] = 1.0
    got = run(t)
    assert torch.allclose(got["final_state"][0, 0], (200.0 + t["dt_bias"][0]) * t["x"][0, -1, 0], rtol=1e-5)
    assert got["final_state"][0, 1] == t["init"][0, 1] and got["final_state"][0, 3] == t["init"][0, 3]
    assert torch.isinf(got["y"][0, 64, 2]) and not torch.isnan(got["y"][0, :64, 2]).any()
    keep = [0, 1, 3, 4, 5, 6, 7]
    for k in ("dx", "ddt"):
        assert torch.isfinite(got[k][..., keep]).all(), k


def test_a_nan_stays_in_its_channel_and_its_future():
    t = make(1, 300, 70, torch.float32, seed=16)
    t["x"][0, 100, 5] = math.nan
    y = run(t)["y"]
    bad = torch.isnan(y)
    assert bad[0, 100:, 5].all() and bad.sum() == 200


def test_gradient_against_differences():
    """Central differences of the 64-bit forward (step 1e-5: truncation about 1e-10, rounding
    1e-11) along random directions; the kernel's gradient is held to its own bound."""
    t = make(2, 90, 33, torch.float32, seed=17, packed=True)
    got = run(t)
    most = reference(t, absolute=True)
    names = {"x": "dx", "dt": "ddt", "dt_bias": "ddt_bias", "A": "dA", "D": "dD", "init": "dinit_state"}

    def loss(s):
        r = reference(s)
        return (r["y"] * t["dy"].double()).sum() + (r["final_state"] * t["dfin"].double()).sum()

    g = torch.Generator(device="cuda").manual_seed(3)
    for k, out in names.items():
        v = torch.randn(t[k].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = dict(t), dict(t)
        up[k], down[k] = t[k].double() + 1e-5 * v, t[k].double() - 1e-5 * v
        diff = (loss(up) - loss(down)) / 2e-5
        along = (got[out].double() * v).sum()
        bound = ((2 * 90 + 32) * 2.0 ** -21 * most[out] * v.abs()).sum() + 1e-6 * diff.abs()
        assert (along - diff).abs() <= bound, f"{k}: {along.item():.9g} against {diff.item():.9g}"


def test_refusals():
    import mamba_ssd_chunked_gb300 as pkg
    t = make(2, 10, 16, torch.float32, seed=18)
    a = (t["dt_bias"], t["A"])
    with pytest.raises(ValueError):
        pkg.ssd_gated_scan(t["x"], t["dt"][:, :9], *a)
    with pytest.raises(ValueError):
        pkg.ssd_gated_scan(t["x"], t["dt"][..., :15].contiguous(), *a)
    with pytest.raises(TypeError):
        pkg.ssd_gated_scan(t["x"], t["dt"].to(torch.bfloat16), *a)
    with pytest.raises(TypeError):
        pkg.ssd_gated_scan(t["x"].half(), t["dt"].half(), *a)
    with pytest.raises(ValueError):
        pkg.ssd_gated_scan(t["x"].cpu(), t["dt"], *a)
    with pytest.raises(ValueError):
        pkg.ssd_gated_scan(t["x"].transpose(1, 2).contiguous().transpose(1, 2), t["dt"], *a)
    with pytest.raises(ValueError):
        pkg.ssd_gated_scan(t["x"], t["dt"], t["dt_bias"], t["A"], init_state=t["init"][:1])
    with pytest.raises(TypeError):
        pkg.ssd_gated_scan(t["x"], t["dt"], *a, seq_idx=torch.zeros(2, 10, dtype=torch.int64, device="cuda"))
    with pytest.raises(pkg.SsdError):
        pkg.ssd_gated_scan(t["x"][:1, :0], t["dt"][:1, :0], *a)  # no tokens
    with pytest.raises(ValueError):
        pkg.ssd_gated_scan_bwd(t["dy"], t["x"], t["dt"], *a, torch.zeros(2, 2, 16, device="cuda"))
    with pytest.raises(ValueError):
        pkg.ssd_gated_scan_step(t["x"][:, 0], t["dt"][:, 0], *a)


def test_a_wait_that_runs_out_is_reported(monkeypatch):
    """With a limit of one nanosecond the tiles of a long sequence do not find what enters them in
    time: the call ends, the device status says so, and the next call is right."""
    import mamba_ssd_chunked_gb300 as pkg
    t = make(1, 60000, 64, torch.float32, seed=19)
    args = (t["x"], t["dt"], t["dt_bias"], t["A"], t["D"])
    want, _, _ = pkg.ssd_gated_scan(*args, init_state=t["init"])
    assert pkg.ssd_device_status() == 0
    monkeypatch.setenv("SSD_DEVICE_WAIT_NS", "1")
    pkg.ssd_gated_scan(*args, init_state=t["init"])
    assert pkg.ssd_device_status() == 4  # SSD_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("SSD_DEVICE_WAIT_NS")
    got, _, _ = pkg.ssd_gated_scan(*args, init_state=t["init"])
    assert pkg.ssd_device_status() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_decays_above_one(io):
    """A of either sign, and zero: forward, gradients and decode steps. delta is below 1.5 and A at most 0.5, so an
    exponent delta A below 0.75 carries delta's 2^-22: a step's decay stays within the 2^-21 of the bound."""
    import mamba_ssd_chunked_gb300 as pkg
    b, L, d = 2, 41, 70
    t = make(b, L, d, DTYPES[io], seed=20)
    t["dt"] = t["dt"].clamp(max=1.0)
    t["dt_bias"] = t["dt_bias"].clamp(max=0.2)
    t["dt_bias"][:8] = 0.2
    t["A"] = torch.linspace(-1.0, 0.05, d, device="cuda")
    t["A"][:6], t["A"][6], t["A"][7] = 0.5, 0.0, 0.1
    check(run(t), t, io)
    ref, most = reference(t), reference(t, absolute=True)
    state = t["init"].clone()
    r = 2.0 ** -8 if io == "bf16" else 2.0 ** -23
    for i in range(L):
        y = pkg.ssd_gated_scan_step(t["x"][:, i], t["dt"][:, i], t["dt_bias"], t["A"], t["D"], state=state)
        bound = (2 * L + 32) * 2.0 ** -21 * most["y"][:, i] + r * ref["y"][:, i].abs()
        assert ((y.double() - ref["y"][:, i]).abs() <= bound).all()
    assert ((state.double() - ref["final_state"]).abs() <= (2 * L + 32) * 2.0 ** -21 * most["final_state"]).all()


def plant(t, row, at, channel, what, value):
    """A copy of t with one entry of x, dt or dy replaced."""
    s = dict(t)
    s[what] = t[what].clone()
    s[what][row, at, channel] = value
    return s


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape,gap", [((2, 700, 70), 90), ((1, 2500, 33), 400), ((2, 130, 64), 1)])
def test_nothing_crosses_packed_sequences(shape, gap, io):
    """Infinities and NaN in one sequence, in its initial state or its final gradient, change nothing in the row's
    other sequences, forward or backward, nor in other channels: bit for bit."""
    b, L, d = shape
    t = make(b, L, d, DTYPES[io], seed=21)
    g = torch.Generator(device="cuda").manual_seed(22)
    cuts = torch.ones(b, L, device="cuda") if gap == 1 else torch.rand(b, L, generator=g, device="cuda") < 1.0 / gap
    cuts[:, [7, 8, 64, L // 2, L - 40]] = 1  # a sequence of one token, the first of a run, one that ends early
    t["seq"] = torch.cumsum(cuts.int(), 1, dtype=torch.int32)
    want = run(t)
    row, c = b - 1, d - 2

    def same(got, first, last, what):
        """Everything but channel c of the sequence at tokens [first, last], and the sums over it."""
        for k in ("y", "dx", "ddt"):
            kept = torch.ones_like(got[k], dtype=torch.bool)
            kept[row, first:last + 1, c] = False
            assert torch.equal(got[k][kept], want[k][kept]), f"{what}: {k}"
        for k, owner in (("final_state", L - 1), ("dinit_state", 0)):
            kept = torch.ones_like(got[k], dtype=torch.bool)
            kept[row, c] = not first <= owner <= last
            assert torch.equal(got[k][kept], want[k][kept]), f"{what}: {k}"
        kept = torch.arange(d, device="cuda") != c
        for k in ("ddt_bias", "dA", "dD"):
            assert torch.equal(got[k][kept], want[k][kept]), f"{what}: {k}"

    seq = t["seq"][row].tolist()
    for at in (0, 6, 7, 8, 63, 64, 70, L // 2 - 1, L // 2, L - 41, L - 40, L - 1):
        first, last = seq.index(seq[at]), L - 1 - seq[::-1].index(seq[at])
        for what, value in (("x", math.inf), ("x", math.nan), ("dt", math.nan), ("dy", -math.inf), ("dy", math.nan)):
            same(run(plant(t, row, at, c, what, value)), first, last, f"{what}[{at}] = {value}")
    for value in (math.inf, math.nan):
        s = dict(t, init=t["init"].clone())
        s["init"][row, c] = value
        same(run(s), 0, L - 1 - seq[::-1].index(seq[0]), f"initial state {value}")
        s = dict(t, dfin=t["dfin"].clone())
        s["dfin"][row, c] = value
        same(run(s), seq.index(seq[-1]), L - 1, f"final gradient {value}")


@pytest.mark.parametrize("vary", [False, True])
def test_slow_decays_in_fp32(vary):
    """Decode steps and the scan of thousands of slow tokens. A decay near one carries 2^-24 (its rounding, and delta's
    2^-22 of an exponent below 2^-8) and a state's update 2^-24, each kept for about T = 1 / (1 - a) tokens; inputs
    are positive, so the state itself bounds the sum: 2^-23 T of it. Gates that vary make the roundings independent: a
    decay's is uniform within 2^-25 and an update's within 2^-24, 2^-24.5 together in the mean square at most, over T / 2
    tokens (a^2 in the place of a): six standard deviations are 6 2^-24.5 sqrt(T / 2)."""
    import mamba_ssd_chunked_gb300 as pkg
    b, L, d = 1, 4000, 96
    t = make(b, L, d, torch.float32, seed=23, with_D=False)
    t["x"], t["init"] = t["x"].abs() + 0.1, t["init"].abs()
    t["dt"] *= 0.1 if vary else 0.0
    slow = torch.linspace(1.0 / 300, 1.0 / 2000, d, device="cuda").double()  # delta |A|, 1 / T
    t["A"] = -torch.ones(d, device="cuda")
    t["dt_bias"] = torch.log(torch.expm1(slow)).float()
    ref = reference(t)["final_state"]
    bound = ref * (6 * 2.0 ** -24.5 * torch.sqrt(0.5 / slow) if vary else 2.0 ** -23 / slow)
    fin = run(t)["final_state"]
    state = t["init"].clone()
    for i in range(L):
        pkg.ssd_gated_scan_step(t["x"][:, i], t["dt"][:, i], t["dt_bias"], t["A"], state=state)
    for what, got in (("scan", fin), ("steps", state)):
        worst = ((got.double() - ref).abs() / bound).max().item()
        assert worst <= 1.0, f"{what}: {worst:.2f} of the bound"


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_infinities_without_a_skip(io):
    """Without D nothing multiplies x or dy but the recurrence: an infinite input gives infinite outputs, as in a decode
    step, where zero times infinity would be NaN."""
    import mamba_ssd_chunked_gb300 as pkg
    t = make(1, 300, 34, DTYPES[io], seed=24, with_D=False)
    t["dt_bias"].fill_(0.0)
    t["A"].fill_(-1e-3)
    t["x"][0, 200, 3], t["dy"][0, 100, 5] = math.inf, -math.inf
    got = run(t)
    assert (got["y"][0, 200:, 3] == math.inf).all() and torch.isfinite(got["y"][0, :200]).all()
    assert (got["dx"][0, :101, 5] == -math.inf).all() and torch.isfinite(got["dx"][0, 101:]).all()
    y = pkg.ssd_gated_scan_step(t["x"][:, 200], t["dt"][:, 200], t["dt_bias"], t["A"], state=t["init"].clone())
    assert y[0, 3] == math.inf
