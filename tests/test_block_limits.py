"""The block operators' largest calls: a launch has fewer than 2^32 threads, so
a call that would need more is refused before anything is enqueued, or goes
out in pieces."""

import pytest
import torch

pytest.importorskip("matrix_aware_optimizer_periodic_amd")
from matrix_aware_optimizer_periodic_amd import binding as bd  # noqa: E402
from test_block_boundary import attn_args, ffn_args, heads, mat, need, needs_lib, norm_args  # noqa: E402

OK, SHAPE = bd.MUON_OK, bd.MUON_E_SHAPE
far = heads(sb=8, sl=8, sh=8)


def attn(**over):
    over = dict(dict(dim=8, causal=0, offset=0, heads=1, kv_heads=1), **over)
    return attn_args(**over, **{n: far for n in ("q", "k", "v", "o", "d_o", "d_q", "d_k", "d_v")})


# (sizes, accepted forward, accepted backward)
@needs_lib
@pytest.mark.parametrize("sizes,fwd,bwd", [
    # 128 rows to a workgroup of 256 threads: 2^24 of them are one too many
    (dict(batch=(1 << 20) - 1, heads=16, kv_heads=16, q_len=128, k_len=0), True, True),
    (dict(batch=1 << 20, heads=16, kv_heads=16, q_len=1, k_len=0), False, False),
    (dict(batch=1 << 19, heads=16, kv_heads=16, q_len=129, k_len=0), False, False),
    (dict(batch=1 << 16, heads=128, kv_heads=1, q_len=255, k_len=0), True, True),
    (dict(batch=1 << 16, heads=128, kv_heads=1, q_len=256, k_len=0), False, False),
    # backward 256 keys to one of 512 threads: 2^23
    (dict(batch=(1 << 20) - 1, heads=8, kv_heads=8, q_len=1, k_len=256), True, True),
    (dict(batch=1 << 20, heads=8, kv_heads=8, q_len=1, k_len=256), True, False),
    (dict(batch=1 << 20, heads=8, kv_heads=8, q_len=1, k_len=1), True, False),
    (dict(batch=1 << 12, heads=1, kv_heads=1, q_len=1, k_len=(1 << 19) - 256), True, True),
    (dict(batch=1 << 12, heads=1, kv_heads=1, q_len=1, k_len=(1 << 19) - 255), True, False),
    # products past 64 bits
    (dict(batch=1 << 20, heads=1 << 30, kv_heads=1 << 30, q_len=1, k_len=1), False, False),
    (dict(batch=1 << 20, heads=1 << 21, kv_heads=1 << 21, q_len=1 << 30, k_len=1 << 30), False, False),
    (dict(batch=1 << 62, heads=4, kv_heads=4, q_len=1, k_len=1), False, False),
])
def test_attention(sizes, fwd, bwd):
    args = attn(**sizes)
    for name, fits in (("muon_attn_fwd", fwd), ("muon_attn_bwd", bwd)):
        assert need(name, args)[0] == (OK if fits else SHAPE), name
    from matrix_aware_optimizer_periodic_amd import block as b
    if not fwd:
        assert b._lib().muon_attn_fwd(args, 0x100000, 1 << 50, None) == SHAPE
    if not bwd:
        assert b._lib().muon_attn_bwd(args, 0x100000, 1 << 50, None) == SHAPE


@needs_lib
@pytest.mark.parametrize("rows,cols,hidden,fits", [
    (1 << 30, 8, 8, True), (1 << 30, 128, 64, True), (1 << 30, 136, 8, False), (1 << 30, 8, 72, False),
    (1 << 27, 128, 15 * 64 - 64, True), (1 << 27, 128, 15 * 64, False),
    (128, 1 << 20, 1 << 15, True), (128, 1 << 20, 1 << 16, False), (128, 1 << 20, 1 << 20, False),
])
def test_feed_forward(rows, cols, hidden, fits):
    args = ffn_args(rows=rows, cols=cols, hidden=hidden)
    for name in ("muon_ffn_fwd", "muon_ffn_bwd"):
        assert need(name, args)[0] == (OK if fits else SHAPE), name


@needs_lib
@pytest.mark.parametrize("rows,group,cols,fits", [
    (0x7fffffff, 0x7fffffff, 8, True), (1 << 31, 1 << 31, 8, False),
    ((1 << 31) - 2, 2, 64, True), (1 << 26, 1, 31 * 64, True), (1 << 26, 1, 32 * 64, False),
])
def test_norm(rows, group, cols, fits):
    vectors = {n: mat(rows // group, cols, 0) for n in ("gate", "scale", "shift", "d_gate", "d_scale", "d_shift")}
    args = norm_args(rows=rows, cols=cols, group=group, **vectors)
    assert need("muon_norm_bwd", args)[0] == (OK if fits else SHAPE)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,per", [((1 << 26) + 77, 8, 4 * (0xffffffff // 256)),
                                           (33_600_000, 257, 0xffffffff // 128)])
def test_norm_rows_in_pieces(rows, cols, per):
    """Four rows to a workgroup of 256 threads, and one to one of 128, a sample
    each: past 2^32 threads both ways.  Rows on both sides of a piece's first
    (`per`) and at the ends equal a small call's."""
    from matrix_aware_optimizer_periodic_amd import block as b
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(rows, 1, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    _, y, stats = b.norm_fwd(x, pre="rms")
    d = b.norm_bwd(None, x, x, None, stats, pre="rms")["resid"]
    for at in (0, rows // 2, per - 20, rows - 40):
        some = slice(at, at + 40)
        _, want, st = b.norm_fwd(x[some], pre="rms")
        assert torch.equal(y[some], want) and torch.equal(stats[some], st), at
        assert torch.equal(d[some], b.norm_bwd(None, x[some], x[some], None, st, pre="rms")["resid"]), at


@pytest.mark.gpu
def test_norm_sums_in_pieces():
    """Modulation of its own for each of 66000 rows of 4096 columns: a workgroup
    of 1024 threads to each 64 columns of a row's sums would be more than 2^32
    threads.  dscale = dy xhat and dshift = dy of each row, dw their sum."""
    from matrix_aware_optimizer_periodic_amd import block as b
    rows, cols = 66_000, 4096
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, 1, cols, generator=gen, device="cuda")
    scale, shift = torch.zeros(rows, cols, device="cuda"), torch.zeros(rows, cols, device="cuda")
    weight = torch.ones(cols, device="cuda")
    how = dict(pre_weight=weight, scale=scale, shift=shift, pre="rms")
    _, y, stats = b.norm_fwd(x, **how)
    dy = torch.randn(rows, 1, cols, generator=gen, device="cuda")
    d = b.norm_bwd(None, dy, x, None, stats, **how)
    assert torch.equal(d["shift"], dy.view(rows, cols))
    for some in (slice(0, 50), slice(65500, 65560), slice(rows - 50, rows)):
        part = dict(pre_weight=weight, scale=scale[some], shift=shift[some], pre="rms")
        want = b.norm_bwd(None, dy[some], x[some], None, stats[some], **part)
        for name in ("scale", "shift", "resid"):
            assert torch.equal(d[name][some], want[name]), name
    # fp32 sums over 66000 rows, 16 threads a column: 4125 additions deep, each
    # off by 2^-24 of a partial sum of random sign
    exact = sum((dy[i:i + 6000].double() * y[i:i + 6000].double()).sum((0, 1)) for i in range(0, rows, 6000))
    assert bool(((d["pre_weight"].double() - exact).abs() <= 4125 * 2.0 ** -24 * exact.abs().max()).all())


@pytest.mark.gpu
def test_norm_sums_of_very_many_samples():
    """A wave to each row's sums: past 2^32 threads from 2^26 rows on."""
    from matrix_aware_optimizer_periodic_amd import block as b
    rows, cols = (1 << 26) + 77, 8
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(rows, 1, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    scale = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    _, _, stats = b.norm_fwd(x, scale=scale, pre="rms")
    d = b.norm_bwd(None, x, x, None, stats, scale=scale, pre="rms")
    for at in (0, rows // 2, 4 * (0xffffffff // 256) - 20, rows - 40):
        some = slice(at, at + 40)
        want = b.norm_bwd(None, x[some], x[some], None, stats[some], scale=scale[some], pre="rms")
        assert torch.equal(d["scale"][some], want["scale"]) and torch.equal(d["resid"][some], want["resid"]), at
