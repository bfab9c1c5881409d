"""GPU checks of the residual update (gate, post-norm, scale, addition, pre-norm)
and its gradients against 64 bits.

Tolerances. Every output is a polynomial in at most 8 fp32 factors and two row
means of `dim` products each; sums are taken in a tree of at most 64 sequential
terms per thread and about 16 levels, 1/rms carries 2^-22, the sigmoid 2^-21. With
M the output's formula on absolute values (both halves of each difference added),

    |got - ref| <= 128 * 2^-23 M + r |ref|

r = 2^-8 for bf16 outputs, 2^-23 for fp32. The weights' gradients add `rows` terms, each
within the same relative distance of its own M, in rows / parts sequential steps
(at most rows): (128 + rows) 2^-23 M.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("y", "residual", "z", "post_weight", "scale", "pre_weight")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_ssd_chunked_gb300 import build
    build.build()


def make(rows, dim, io, res, seed, drop=()):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    t = {"y": n(rows, dim).to(io), "z": n(rows, dim).to(io), "residual": (2 * n(rows, dim)).to(res),
         "post_weight": 1 + 0.1 * n(dim), "scale": 0.5 + 0.1 * n(dim), "pre_weight": 1 + 0.1 * n(dim),
         "dout": n(rows, dim).to(io), "dres": n(rows, dim).to(res)}
    for k in drop:
        t[k] = None
    if t["pre_weight"] is None:
        t["dout"] = None
    return t


def reference(t, eps=EPS, absolute=False):
    """The formulas in 64 bits; `absolute`: on absolute values, differences as sums
    (the norms' 1/rms keep their values)."""
    sign = 1.0 if absolute else -1.0
    f = lambda v: None if v is None else (v.double().abs() if absolute else v.double())
    y, z, res, post, scale, pre, dout, dres = (f(t[k]) for k in
                                               ("y", "z", "residual", "post_weight", "scale", "pre_weight", "dout", "dres"))
    one = torch.ones((), dtype=torch.float64, device=y.device)
    zr = None if t["z"] is None else t["z"].double()
    sig = None if zr is None else torch.sigmoid(zr)
    gate = one if zr is None else (zr * sig).abs() if absolute else zr * sig
    u = y * gate
    real = reference(t, eps)["_rho"] if absolute else None
    rho_u = real[0] if absolute else (torch.rsqrt((u * u).mean(1, keepdim=True) + eps) if post is not None else one)
    un = u * rho_u
    c = (one if post is None else post) * (one if scale is None else scale)
    r = c * un + (0 if res is None else res)
    rho = real[1] if absolute else torch.rsqrt((r * r).mean(1, keepdim=True) + eps)
    rn = r * rho
    out = {"residual_out": r, "_rho": (rho_u, rho)}
    if pre is not None:
        out["out"] = rn * pre
    dr = torch.zeros_like(r) if dres is None else dres
    if pre is not None:
        n = dout * pre
        dr = dr + rho * (n + sign * rn * (n * rn).mean(1, keepdim=True))
    e = dr * c
    du = rho_u * (e + sign * un * (e * un).mean(1, keepdim=True)) if post is not None else e
    out["dy"] = du * gate
    if zr is not None:
        slope = sig * (1 + zr.abs() * (1 - sig)) if absolute else sig * (1 + zr * (1 - sig))
        out["dz"] = du * y * slope
    if res is not None:
        out["dresidual"] = dr
    both = (dr * un).sum(0)
    if post is not None:
        out["dpost_weight"] = both * (one if scale is None else scale)
    if scale is not None:
        out["dscale"] = both * (one if post is None else post)
    if pre is not None:
        out["dpre_weight"] = (dout * rn).sum(0)
    return out


def run(t, eps=EPS, **kw):
    import mamba_ssd_chunked_gb300 as pkg
    a = {k: t[k] for k in NAMES[1:]}
    res_out, out, rstd = pkg.ssd_block_norm(t["y"], eps=eps, return_rstd=True, **a, **kw)
    if t["residual"] is None:
        kw = dict(kw)
    g = pkg.ssd_block_norm_bwd(t["dout"], t["dres"], t["y"], rstd, **a, **kw)
    torch.cuda.synchronize()
    got = {"residual_out": res_out, "out": out}
    got.update(zip(("dy", "dresidual", "dz", "dpost_weight", "dscale", "dpre_weight"), g))
    return {k: v for k, v in got.items() if v is not None}


def check(got, t, eps=EPS, what=""):
    ref, most = reference(t, eps), reference(t, eps, absolute=True)
    assert set(got) == {k for k in ref if k != "_rho"}, what
    rows = t["y"].reshape(-1, t["y"].shape[-1]).shape[0]
    for k, v in got.items():
        r = 2.0 ** -8 if v.dtype == torch.bfloat16 else 2.0 ** -23
        n = 128 + (rows if k.endswith("weight") or k == "dscale" else 0)
        off = ((v.double() - ref[k]).abs() - n * 2.0 ** -23 * most[k] - r * ref[k].abs()).max().item()
        assert off <= 0, f"{what} {k}: {off:.3e} over the bound"


TYPES = [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")]
# one element; odd widths; a warp's width; several vectors per thread; the widest row
SHAPES = [(1, 1), (5, 7), (3, 64), (9, 100), (33, 257), (70, 771), (1, 768), (130, 2560), (17, 4100), (5, 8192),
          (3, 9001), (2, 16384), (700, 40)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_the_formulas(shape, types):
    t = make(*shape, DT[types[0]], DT[types[1]], seed=sum(shape))
    check(run(t), t, what=f"{shape} {types}")


@pytest.mark.parametrize("drop", [("z",), ("residual",), ("post_weight",), ("scale",), ("pre_weight",), ("dres",),
                                  ("z", "post_weight", "scale"), ("z", "residual", "scale", "dres"),
                                  ("z", "residual", "post_weight"), ("pre_weight", "z", "scale")])
@pytest.mark.parametrize("types", TYPES)
def test_absent_inputs(drop, types):
    t = make(21, 96, DT[types[0]], DT[types[1]], seed=3, drop=drop)
    kw = {"residual_dtype": DT[types[1]]} if t["residual"] is None else {}
    check(run(t, **kw), t, what=str(drop))


@pytest.mark.parametrize("dim", [4096, 4095, 16384])
def test_offsets_past_32_bits(dim):
    """More than 2^31 elements (both persistent kernels, and the direct ones): the first and the last rows."""
    rows = 2 ** 31 // dim + 300
    g = torch.Generator(device="cuda").manual_seed(15)
    t = make(4, dim, torch.bfloat16, torch.bfloat16, seed=16)
    for k in ("y", "z", "residual", "dout", "dres"):
        t[k] = torch.randn(rows, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    got = run(t)
    for part in (slice(0, 64), slice(rows - 64, rows)):
        s = {k: v[part] if v.dim() == 2 else v for k, v in t.items()}
        ref = reference(s)  # the weights' gradients add up all rows: not compared here
        sums = {k: ref[k] for k in ("dpost_weight", "dscale", "dpre_weight")}
        check({k: sums[k] if k in sums else got[k][part] for k in got}, s, what=f"rows {part}")


def test_zero_rows_and_zero_eps():
    t = make(6, 128, torch.float32, torch.float32, seed=4)
    t["y"][2] = 0
    t["y"][3] = 0
    t["residual"][3] = 0
    got = run(t)
    check(got, t)
    assert all(torch.isfinite(v).all() for v in got.values())
    t = make(6, 128, torch.float32, torch.float32, seed=5)
    check(run(t, eps=0.0), t, eps=0.0)


def test_large_and_small_rows():
    """Rows whose squares reach 2^100 and 2^-60 (below eps): still inside fp32."""
    t = make(4, 256, torch.float32, torch.float32, seed=6)
    t["residual"][0] *= 2.0 ** 49
    t["y"][1] *= 2.0 ** 40
    t["residual"][2] *= 2.0 ** -30
    t["y"][2] *= 2.0 ** -30
    check(run(t), t)


def test_saturated_gates():
    t = make(4, 64, torch.bfloat16, torch.float32, seed=7)
    t["z"][0], t["z"][1], t["z"][2, ::2] = 300.0, -300.0, -1e30
    got = run(t)
    assert all(torch.isfinite(v).all() for v in got.values())
    # silu(-300) is below fp32's range: row 1's un and its gradients are exactly zero
    # there, and the residual passes unchanged
    assert torch.equal(got["residual_out"][1], t["residual"][1])
    assert (got["dy"][1] == 0).all() and (got["dz"][1] == 0).all()
    # silu(300) = 300 and its slope 1: the row is the plain norm of 300 y
    one = {k: (v if v is None or v.dim() == 1 else v[:1]) for k, v in t.items()}
    one.update(z=None, y=t["y"][:1].float() * 300, dout=one["dout"].float())
    ref = reference(one)
    for k in ("residual_out", "dresidual"):
        assert torch.allclose(got[k][:1].double(), ref[k], rtol=1e-5, atol=1e-5), k


def test_a_nan_stays_in_its_row():
    t = make(5, 300, torch.float32, torch.float32, seed=8)
    t["y"][2, 17] = math.nan
    got = run(t)
    for k in ("residual_out", "out", "dy", "dz", "dresidual"):
        bad = torch.isnan(got[k]).any(1)
        assert bad.tolist() == [False, False, True, False, False], k


@pytest.mark.parametrize("offset", [0, 3, 8])
def test_slices_and_leading_dimensions(offset):
    t = make(24, 64, torch.bfloat16, torch.float32, seed=9)
    want = run(t)
    wide = torch.zeros(4, 6, 3 * 64 + 16, dtype=torch.bfloat16, device="cuda")
    s = {k: (v.reshape(4, 6, 64) if v is not None and v.dim() == 2 else v) for k, v in t.items()}
    for i, k in enumerate(("y", "z", "dout")):
        wide[..., offset + 64 * i:offset + 64 * (i + 1)] = s[k]
        s[k] = wide[..., offset + 64 * i:offset + 64 * (i + 1)]
    got = run(s)
    ref, most = reference(t), reference(t, absolute=True)
    for k in want:
        assert got[k].shape == ((4, 6, 64) if want[k].dim() == 2 else want[k].shape)
    check({k: v.reshape(want[k].shape) for k, v in got.items()}, t)


def test_runs_repeat_bit_for_bit_and_on_another_stream():
    t = make(3000, 320, torch.bfloat16, torch.float32, seed=10)
    first = run(t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for again in (run(t), run(t, stream=s.cuda_stream)):
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(first[k], again[k]), k


def test_gradient_against_differences():
    """Central differences of the 64-bit forward (step 1e-5) along random directions."""
    t = make(11, 40, torch.float32, torch.float32, seed=11)
    got, most = run(t), reference(t, absolute=True)

    def loss(s):
        r = reference(s)
        return (r["out"] * t["dout"].double()).sum() + (r["residual_out"] * t["dres"].double()).sum()

    g = torch.Generator(device="cuda").manual_seed(3)
    for k in NAMES:
        v = torch.randn(t[k].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = dict(t), dict(t)
        up[k], down[k] = t[k].double() + 1e-5 * v, t[k].double() - 1e-5 * v
        diff = (loss(up) - loss(down)) / 2e-5
        along = (got["d" + k].double() * v).sum()
        bound = ((128 + 11) * 2.0 ** -23 * most["d" + k] * v.abs()).sum() + 1e-6 * (1 + diff.abs())
        assert (along - diff).abs() <= bound, f"{k}: {along.item():.9g} against {diff.item():.9g}"


def test_agrees_with_the_gated_norm():
    """Without a residual, the norm after a block is the framework's gated RMSNorm."""
    import mamba_ssd_chunked_gb300 as pkg
    t = make(40, 512, torch.float32, torch.float32, seed=12)
    r, out, _ = pkg.ssd_block_norm(t["y"], z=t["z"], post_weight=t["post_weight"], eps=EPS)
    assert out is None
    want = pkg.ssd_gated_rmsnorm(t["y"], t["z"], t["post_weight"], eps=EPS)
    assert torch.allclose(r, want, rtol=1e-5, atol=1e-6)


def test_refusals():
    import mamba_ssd_chunked_gb300 as pkg
    t = make(4, 32, torch.float32, torch.float32, seed=13)
    with pytest.raises(TypeError):
        pkg.ssd_block_norm(t["y"].half())
    with pytest.raises(TypeError):
        pkg.ssd_block_norm(t["y"], z=t["z"].bfloat16())
    with pytest.raises(ValueError):
        pkg.ssd_block_norm(t["y"], residual=t["residual"][:3])
    with pytest.raises(ValueError):
        pkg.ssd_block_norm(t["y"], post_weight=t["post_weight"][:31])
    with pytest.raises(ValueError):
        pkg.ssd_block_norm(t["y"].t())
    with pytest.raises(ValueError):
        pkg.ssd_block_norm(t["y"].cpu())
    with pytest.raises(pkg.SsdError):
        pkg.ssd_block_norm(t["y"], eps=-1.0)
    with pytest.raises(pkg.SsdError):
        pkg.ssd_block_norm(t["y"], residual=t["residual"].bfloat16())  # fp32 io takes an fp32 residual
    with pytest.raises(pkg.SsdError):
        pkg.ssd_block_norm(torch.zeros(1, 16385, device="cuda"))
    _, _, rstd = pkg.ssd_block_norm(t["y"], residual=t["residual"], pre_weight=t["pre_weight"], return_rstd=True)
    with pytest.raises(ValueError):
        pkg.ssd_block_norm_bwd(None, t["dres"], t["y"], rstd, residual=t["residual"], pre_weight=t["pre_weight"])
    with pytest.raises(ValueError):
        pkg.ssd_block_norm_bwd(t["dout"], t["dres"], t["y"], rstd[:3], residual=t["residual"],
                               pre_weight=t["pre_weight"])
    with pytest.raises(pkg.SsdError):
        pkg.ssd_block_norm_bwd(None, None, t["y"], rstd, residual=t["residual"])


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("shape", [(3100, 129), (3100, 771), (1300, 2559), (700, 4095), (700, 5119), (1500, 768), (800, 4096)])
def test_many_rows(shape, types):
    """Enough rows for the persistent kernels, on and off 16-byte row starts."""
    t = make(*shape, DT[types[0]], DT[types[1]], seed=sum(shape))
    check(run(t), t, what=f"{shape} {types}")


def test_many_rows_inside_wider_ones():
    """Rows that start on every multiple of two bytes, some at the very start and end of their allocation."""
    rows, dim = 2000, 200
    t = make(rows, dim, torch.bfloat16, torch.float32, seed=14)
    want = run(t)
    for pad, offset in ((1, 0), (1, 1), (3, 2), (8, 8)):
        s = dict(t)
        for k in ("y", "z", "dout"):
            wide = torch.full((rows, dim + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
            wide[:, offset:offset + dim] = t[k]
            s[k] = wide[:, offset:offset + dim]
        check(run(s), t, what=f"pad {pad} offset {offset}")
        for k in ("residual_out", "out"):
            assert torch.allclose(run(s)[k].float(), want[k].float(), rtol=1e-2, atol=1e-5), k


@pytest.mark.parametrize("drop", [("pre_weight",), ("pre_weight", "scale"), ("pre_weight", "z", "residual"), ("post_weight",),
                                  ("z", "residual", "post_weight", "scale"), ("residual", "scale", "pre_weight", "dres")])
@pytest.mark.parametrize("shape", [(2000, 2560), (1300, 2559), (3100, 768), (3100, 771)])
def test_many_rows_with_absent_inputs(shape, drop):
    """The persistent kernels with several warps per row, in the forms that leave sums and their barriers out: right,
    and the same bits every time."""
    t = make(*shape, torch.bfloat16, torch.float32, seed=sum(shape), drop=drop)
    if t["dout"] is None and t["dres"] is None:
        import mamba_ssd_chunked_gb300 as pkg
        a = {k: t[k] for k in NAMES[1:]}
        again = lambda: {"residual_out": pkg.ssd_block_norm(t["y"], eps=EPS, **a)[0]}
        ref, most = reference({**t, "dres": t["y"].float()}), reference({**t, "dres": t["y"].float()}, absolute=True)
        off = (again()["residual_out"].double() - ref["residual_out"]).abs() - 129 * 2.0 ** -23 * most["residual_out"]
        assert off.max().item() <= 0
    else:
        again = lambda: run(t)
        check(again(), t, what=f"{shape} {drop}")
    first = again()
    for _ in range(10):
        got = again()
        for k in first:
            assert torch.equal(first[k], got[k]), k


@pytest.mark.parametrize("shape", [(3000, 2560), (3000, 2559)])
def test_a_wait_that_runs_out_is_reported(shape, monkeypatch):
    """With a limit of one nanosecond the persistent kernels do not see their rows arrive in time: the calls end, the
    device status says so, and the next ones are right."""
    import mamba_ssd_chunked_gb300 as pkg
    t = make(*shape, torch.bfloat16, torch.float32, seed=17)
    want = run(t)
    assert pkg.ssd_device_status() == 0
    monkeypatch.setenv("SSD_DEVICE_WAIT_NS", "1")
    run(t)
    assert pkg.ssd_device_status() == 4  # SSD_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("SSD_DEVICE_WAIT_NS")
    got = run(t)
    assert pkg.ssd_device_status() == 0
    for k in want:
        assert torch.equal(want[k], got[k]), k
