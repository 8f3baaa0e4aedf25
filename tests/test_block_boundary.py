"""The transformer-block operators' C ABI and bindings on the CPU: the library
exports what include/muon_block.h declares, the packed argument structures
have the header's size and layout, and every bad argument is refused with its
status before anything is enqueued.  Nothing here launches a kernel."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

m = pytest.importorskip("matrix_aware_optimizer_periodic_amd")
from matrix_aware_optimizer_periodic_amd import binding as bd  # noqa: E402
from matrix_aware_optimizer_periodic_amd import block as b  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "muon_block.h")
CSRC = os.path.join(ROOT, "matrix_aware_optimizer_periodic_amd", "csrc")
HAVE_LIB = os.path.exists(bd.LIB_PATH)
needs_lib = pytest.mark.skipif(not HAVE_LIB, reason="libmuon_hip.so not built")
FAKE = 0x100000          # an aligned stand-in address, never dereferenced by validation


def test_header_and_binding_name_the_same_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"^\s*(?:const char\*|muon_status)\s+(muon_\w+)\s*\(", text, re.M))
    assert declared == set(b.BLOCK_EXPORTED)
    if HAVE_LIB:
        for name in declared:
            assert hasattr(m.lib(), name), name


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_packed_structures_match_the_header(tmp_path):
    """Sizes and a field's offset near each end, from the compiler."""
    src = tmp_path / "s.cpp"
    src.write_text('#include "muon_block.h"\n#include <cstdio>\nint main() { printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu\\n",'
                   "sizeof(muon_norm_args), offsetof(muon_norm_args, stats), offsetof(muon_norm_args, d_pre_weight),"
                   "sizeof(muon_attn_args), offsetof(muon_attn_args, q_lens), offsetof(muon_attn_args, d_v),"
                   "sizeof(muon_ffn_args), offsetof(muon_ffn_args, x), offsetof(muon_ffn_args, d_w_down)); }\n")
    exe = tmp_path / "s"
    subprocess.run(["g++", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    head = ctypes.sizeof(bd.MuonTensor)
    assert head == 40
    n, a, f = b.NORM_ARGS.size, b.ATTN_ARGS.size, b.FFN_ARGS.size
    assert got == [n, 40 + 9 * head, n - head, a, 24 + 4 * 4 + 8 + 4 + 4, a - 32, f, 32, f - head]


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_fast_division_is_exact(tmp_path):
    src = tmp_path / "d.cpp"
    src.write_text("""
#include "block_internal.h"
#include <cstdio>
#include <cstdlib>
using namespace muon;
int main() {
  unsigned long bad = 0;
  const uint32_t big[] = {1u << 20, (1u << 20) + 1, (1u << 30) - 1, 1u << 30, 0x7fffffffu};
  for (uint32_t i = 0; i < 5205; ++i) {
    const uint32_t d = i < 5200 ? i + 1 : big[i - 5200];
    const FastDiv f = fast_div(d);
    for (uint32_t j = 0; j < 200; ++j) {
      uint64_t n = j < 20 ? j : j < 100 ? uint64_t(d) * j + (j & 1 ? 0 : d - 1) : j == 100 ? 0x7fffffffu : uint32_t(rand());
      n &= 0x7fffffffu;
      const uint32_t q = (uint32_t((n * f.mul) >> 32) + uint32_t(n)) >> f.shift;
      bad += q != n / d;
    }
  }
  fast_div(0);
  printf("bad %lu\\n", bad);
}
""")
    exe = tmp_path / "d"
    subprocess.run(["g++", "-O1", "-D__HIP_PLATFORM_AMD__", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I",
                    CSRC, "-I", "/opt/rocm/include", str(src), "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "bad 0" in r.stdout, r.stdout + r.stderr


# ------------------------------------------------------------ C refusals
def mat(rows, cols, dt=1, ptr=FAKE, ld=None, reserved=0):
    return [ptr, rows, cols, cols if ld is None else ld, dt, reserved]


NONE = [0] * 6


def norm_args(**over):
    """Arguments of a valid backward call (which hold the forward's too)."""
    v = dict(rows=32, cols=64, group=8, post=1, pre=2, alpha=1.0, eps=1e-6, resid=mat(32, 64, 0), h=mat(32, 64),
             resid_out=mat(32, 64, 0), y=mat(32, 64), gate=mat(4, 64, 0), scale=mat(4, 64, 0), shift=mat(4, 64, 0),
             post_weight=mat(1, 64, 0), pre_weight=mat(1, 64, 0), stats=FAKE, d_resid_out=mat(32, 64, 0),
             d_y=mat(32, 64), d_resid=mat(32, 64, 0), d_h=mat(32, 64), d_gate=mat(4, 64, 0), d_scale=mat(4, 64, 0),
             d_shift=mat(4, 64, 0), d_post_weight=mat(1, 64, 0), d_pre_weight=mat(1, 64, 0))
    v.update(over)
    order = ("resid", "h", "resid_out", "y", "gate", "scale", "shift", "post_weight", "pre_weight")
    back = ("d_resid_out", "d_y", "d_resid", "d_h", "d_gate", "d_scale", "d_shift", "d_post_weight", "d_pre_weight")
    return b.NORM_ARGS.pack(v["rows"], v["cols"], v["group"], v["post"], v["pre"], v["alpha"], v["eps"],
                            *sum((v[k] for k in order), []), v["stats"], *sum((v[k] for k in back), []))


def need(name, args):
    n = ctypes.c_size_t(0)
    st = getattr(b._lib(), name + "_workspace")(args, n)
    return st, n.value


E = bd


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(cols=0), E.MUON_E_SHAPE), (dict(cols=16385), E.MUON_E_SHAPE), (dict(rows=-1), E.MUON_E_SHAPE),
    (dict(group=0), E.MUON_E_SHAPE), (dict(group=5), E.MUON_E_SHAPE), (dict(post=3), E.MUON_E_ARG),
    (dict(pre=-1), E.MUON_E_ARG), (dict(alpha=float("nan")), E.MUON_E_ARG), (dict(eps=-1.0), E.MUON_E_ARG),
    (dict(gate=mat(3, 64)), E.MUON_E_SHAPE), (dict(scale=mat(4, 64, 2)), E.MUON_E_DTYPE),
    (dict(shift=mat(4, 64, ld=63)), E.MUON_E_ALIGN), (dict(post_weight=mat(2, 64)), E.MUON_E_SHAPE),
    (dict(stats=0), E.MUON_E_ARG), (dict(stats=FAKE + 4), E.MUON_E_ALIGN), (dict(h=NONE), E.MUON_E_ARG),
    (dict(h=mat(32, 64, reserved=1)), E.MUON_E_SHAPE), (dict(h=mat(32, 64, ptr=FAKE + 1)), E.MUON_E_ALIGN),
])
def test_norm_refuses_both_ways(over, status):
    args = norm_args(**over)
    assert b._lib().muon_norm_fwd(args, None) == status
    assert b._lib().muon_norm_bwd(args, FAKE, 1 << 30, None) == status
    assert b._lib().muon_block_last_error()


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(resid=NONE), E.MUON_E_ARG), (dict(resid=mat(31, 64, 0)), E.MUON_E_SHAPE),
    (dict(resid_out=mat(32, 64, 1)), E.MUON_E_DTYPE), (dict(y=mat(32, 64, 0)), E.MUON_E_DTYPE),
    (dict(y=NONE), E.MUON_E_ARG), (dict(resid=mat(32, 64, 0, ld=1 << 23)), E.MUON_E_ALIGN),
])
def test_norm_fwd_refuses(over, status):
    assert b._lib().muon_norm_fwd(norm_args(**over), None) == status


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(d_resid=NONE), E.MUON_E_ARG), (dict(d_h=NONE), E.MUON_E_ARG), (dict(d_y=NONE), E.MUON_E_ARG),
    (dict(d_h=mat(32, 64, 0)), E.MUON_E_DTYPE), (dict(d_resid_out=mat(32, 64, 1)), E.MUON_E_DTYPE),
    (dict(resid_out=NONE), E.MUON_E_ARG), (dict(d_gate=mat(4, 64, 1)), E.MUON_E_DTYPE),
    (dict(d_pre_weight=mat(4, 64, 0)), E.MUON_E_SHAPE), (dict(rows=0), E.MUON_E_SHAPE),
])
def test_norm_bwd_refuses(over, status):
    assert b._lib().muon_norm_bwd(norm_args(**over), FAKE, 1 << 30, None) == status


@needs_lib
def test_norm_workspace():
    st, n = need("muon_norm_bwd", norm_args())
    assert st == E.MUON_OK and n >= 4 * 3 * 64 * 4 + 4 * 2 * 64 * 4
    L = b._lib()
    assert L.muon_norm_bwd(norm_args(), FAKE, n - 1, None) == E.MUON_E_WORKSPACE
    assert L.muon_norm_bwd(norm_args(), None, n, None) == E.MUON_E_WORKSPACE
    assert L.muon_norm_bwd(norm_args(), FAKE + 128, n, None) == E.MUON_E_ALIGN
    none = {k: NONE for k in ("d_gate", "d_scale", "d_shift", "d_post_weight", "d_pre_weight")}
    assert need("muon_norm_bwd", norm_args(**none)) == (E.MUON_OK, 0)
    assert L.muon_norm_bwd_workspace(norm_args(), None) == E.MUON_E_ARG
    assert L.muon_norm_fwd(norm_args(rows=0, group=1, gate=NONE, scale=NONE, shift=NONE), None) == E.MUON_OK


def heads(ptr=FAKE, sb=1 << 16, sl=512, sh=64):
    return [ptr, sb, sl, sh]


def attn_args(**over):
    v = dict(batch=2, q_len=100, k_len=120, heads=8, kv_heads=4, dim=64, causal=1, offset=20, scale=0.125, reserved=0,
             q_lens=0, k_lens=0, q=heads(), k=heads(), v=heads(), o=heads(), lse=FAKE, d_o=heads(), d_q=heads(),
             d_k=heads(), d_v=heads())
    v.update(over)
    return b.ATTN_ARGS.pack(*(v[k] for k in ("batch", "q_len", "k_len", "heads", "kv_heads", "dim", "causal", "offset",
                                             "scale", "reserved", "q_lens", "k_lens")),
                            *v["q"], *v["k"], *v["v"], *v["o"], v["lse"], *v["d_o"], *v["d_q"], *v["d_k"], *v["d_v"])


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), E.MUON_E_SHAPE), (dict(q_len=-1), E.MUON_E_SHAPE), (dict(heads=0), E.MUON_E_SHAPE),
    (dict(kv_heads=3), E.MUON_E_SHAPE), (dict(dim=60), E.MUON_E_SHAPE), (dict(dim=136), E.MUON_E_SHAPE),
    (dict(dim=0), E.MUON_E_SHAPE), (dict(causal=2), E.MUON_E_ARG), (dict(reserved=1), E.MUON_E_ARG),
    (dict(scale=0.0), E.MUON_E_ARG), (dict(scale=-1.0), E.MUON_E_ARG), (dict(scale=float("inf")), E.MUON_E_ARG),
    (dict(q_len=1 << 31), E.MUON_E_SHAPE), (dict(batch=1 << 21), E.MUON_E_SHAPE),
    (dict(q=heads(ptr=0)), E.MUON_E_ARG), (dict(k=heads(ptr=FAKE + 8)), E.MUON_E_ALIGN),
    (dict(v=heads(sl=516)), E.MUON_E_ALIGN), (dict(q=heads(sb=-8)), E.MUON_E_SHAPE),
    (dict(k=heads(sl=1 << 23)), E.MUON_E_SHAPE), (dict(o=heads(ptr=0)), E.MUON_E_ARG), (dict(lse=0), E.MUON_E_ARG),
])
def test_attention_refuses_both_ways(over, status):
    args = attn_args(**over)
    assert b._lib().muon_attn_fwd(args, FAKE, 1 << 40, None) == status
    assert b._lib().muon_attn_bwd(args, FAKE, 1 << 40, None) == status
    assert b._lib().muon_block_last_error()


@needs_lib
@pytest.mark.parametrize("over", [dict(d_o=heads(ptr=0)), dict(d_q=heads(ptr=0)), dict(d_k=heads(ptr=0)),
                                  dict(d_v=heads(ptr=0))])
def test_attention_bwd_refuses_missing_gradients(over):
    assert b._lib().muon_attn_bwd(attn_args(**over), FAKE, 1 << 40, None) == E.MUON_E_ARG


@needs_lib
def test_attention_workspace_and_empty():
    L = b._lib()
    st, n = need("muon_attn_bwd", attn_args())
    assert st == E.MUON_OK and n >= 2 * 2 * 8 * 100 * 4
    assert L.muon_attn_bwd(attn_args(), FAKE, n - 1, None) == E.MUON_E_WORKSPACE
    # one query over many keys is split along the keys and needs room for the parts
    few = dict(q_len=1, k_len=9000)
    st, n = need("muon_attn_fwd", attn_args(**few))
    assert st == E.MUON_OK and n > 0
    assert L.muon_attn_fwd(attn_args(**few), FAKE, n - 1, None) == E.MUON_E_WORKSPACE
    for empty in (dict(batch=0), dict(q_len=0), dict(q_len=0, k_len=0)):
        assert need("muon_attn_fwd", attn_args(**empty))[0] == E.MUON_OK
        assert L.muon_attn_fwd(attn_args(**empty), None, 0, None) == E.MUON_OK
    assert L.muon_attn_bwd(attn_args(q_len=0, k_len=0), None, 0, None) == E.MUON_OK
    assert need("muon_attn_bwd", attn_args(k_len=0))[0] == E.MUON_OK


def ffn_args(**over):
    v = dict(rows=40, cols=64, hidden=96, act=0, reserved=0, x=mat(40, 64), y=mat(40, 64), w_gate=mat(96, 64),
             w_up=mat(96, 64), w_down=mat(64, 96), gu=mat(40, 192), d_y=mat(40, 64), d_x=mat(40, 64),
             d_w_gate=mat(96, 64, 0), d_w_up=mat(96, 64, 0), d_w_down=mat(64, 96, 0))
    v.update(over)
    order = ("x", "y", "w_gate", "w_up", "w_down", "gu", "d_y", "d_x", "d_w_gate", "d_w_up", "d_w_down")
    return b.FFN_ARGS.pack(v["rows"], v["cols"], v["hidden"], v["act"], v["reserved"], *sum((v[k] for k in order), []))


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), E.MUON_E_SHAPE), (dict(cols=60), E.MUON_E_SHAPE), (dict(hidden=0), E.MUON_E_SHAPE),
    (dict(hidden=(1 << 20) + 8), E.MUON_E_SHAPE), (dict(act=2), E.MUON_E_ARG), (dict(reserved=1), E.MUON_E_ARG),
    (dict(x=NONE), E.MUON_E_ARG), (dict(x=mat(41, 64)), E.MUON_E_SHAPE), (dict(x=mat(40, 64, 0)), E.MUON_E_DTYPE),
    (dict(x=mat(40, 64, ld=66)), E.MUON_E_ALIGN), (dict(x=mat(40, 64, ptr=FAKE + 8)), E.MUON_E_ALIGN),
    (dict(w_gate=mat(64, 96)), E.MUON_E_SHAPE), (dict(w_up=NONE), E.MUON_E_ARG),
    (dict(w_down=mat(64, 96, 0)), E.MUON_E_DTYPE), (dict(gu=mat(40, 96)), E.MUON_E_SHAPE),
])
def test_ffn_refuses_both_ways(over, status):
    args = ffn_args(**over)
    assert b._lib().muon_ffn_fwd(args, FAKE, 1 << 40, None) == status
    assert b._lib().muon_ffn_bwd(args, FAKE, 1 << 40, None) == status


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(rows=0), E.MUON_E_SHAPE), (dict(gu=NONE), E.MUON_E_ARG), (dict(d_y=NONE), E.MUON_E_ARG),
    (dict(d_x=mat(40, 64, 0)), E.MUON_E_DTYPE), (dict(d_w_up=mat(96, 64, 1)), E.MUON_E_DTYPE),
    (dict(d_w_down=mat(96, 64, 0)), E.MUON_E_SHAPE), (dict(d_w_gate=mat(96, 64, 0, ld=65)), E.MUON_E_ALIGN),
])
def test_ffn_bwd_refuses(over, status):
    assert b._lib().muon_ffn_bwd(ffn_args(**over), FAKE, 1 << 40, None) == status


@needs_lib
def test_ffn_workspace():
    L = b._lib()
    for name, least in (("muon_ffn_fwd", 40 * 96 * 2), ("muon_ffn_bwd", 3 * 40 * 96 * 2)):
        st, n = need(name, ffn_args())
        assert st == E.MUON_OK and n >= least
        assert getattr(L, name)(ffn_args(), FAKE, n - 1, None) == E.MUON_E_WORKSPACE
        assert getattr(L, name)(ffn_args(), FAKE + 16, n, None) == E.MUON_E_ALIGN
    assert L.muon_ffn_fwd(ffn_args(rows=0), None, 0, None) == E.MUON_OK


@needs_lib
def test_null_arguments():
    L = b._lib()
    for name in b.BLOCK_EXPORTED[1:]:
        f = getattr(L, name)
        n = ctypes.c_size_t(0)
        st = f(None, n) if name.endswith("_workspace") else f(None, None) if name == "muon_norm_fwd" else f(None, None, 0, None)
        assert st == E.MUON_E_ARG, name


# ------------------------------------------------------- Python refusals
def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        m.norm_fwd(x)
    with pytest.raises(ValueError, match="GPU"):
        m.attn_fwd(x.view(1, 4, 1, 64), x.view(1, 4, 1, 64), x.view(1, 4, 1, 64))
    with pytest.raises(ValueError, match="GPU"):
        m.ffn_fwd(x, w, w, w.T)


def test_matrix_descriptors():
    x = torch.zeros(6, 40)
    assert b._mat(x, 6, 40)[1:] == (6, 40, 40, 0, 0)
    assert b._mat(x[:, 8:24], 6, 16)[1:] == (6, 16, 40, 0, 0)
    assert b._mat(x.view(2, 3, 40)[:, :, :8], 6, 8)[1:] == (6, 8, 40, 0, 0)
    assert b._mat(x[:1, 4:9], 1, 5)[3] == 5
    for bad in (x.T, x.view(2, 3, 40)[:, :2], x[::2].view(3, 2, 20)[:, 0]):
        if bad.shape[-1] == 20:
            continue
        with pytest.raises(ValueError):
            b._mat(bad, bad.shape[:-1].numel(), bad.shape[-1])
    with pytest.raises(ValueError):
        b._mat(torch.zeros(1, 40).expand(6, 40), 6, 40)      # rows on top of each other
    with pytest.raises(ValueError):
        b._mat(x, 5, 40)
    with pytest.raises(TypeError):
        b._mat(x.half(), 6, 40)


def test_names_are_reached_through_the_package():
    for n in ("norm_fwd", "norm_bwd", "residual_norm", "attn_fwd", "attn_bwd", "attention", "ffn_fwd", "ffn_bwd",
              "gated_ffn"):
        assert callable(getattr(m, n))
    with pytest.raises(AttributeError):
        m.no_such_operator
