"""C-ABI checks of include/ipttt_block.h that need no GPU: exports, structure layouts,
workspace sizes, and every refusal, before any device work (the pointers are host
memory)."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

from chunked_weight_mlp_amd import block as K
from chunked_weight_mlp_amd import build as bld
from chunked_weight_mlp_amd import ipttt as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ipttt_block.h")
LLVM = "/opt/rocm/llvm/bin"


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.fail("libipttt.so is not built: run __graft_entry__.build()")
    return K.load()


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(ipttt_[a-z_]+)\s*\(", text)))


def test_header_declares_the_binding_exports(lib):
    assert declared_functions() == sorted(K.EXPORTS)
    for f in declared_functions():
        assert hasattr(lib, f)


def test_structure_layouts_match_c(tmp_path):
    structs = {"ipttt_norm_desc": K.NormDesc, "ipttt_view": K.View, "ipttt_recurrence": K.RecurrenceDesc,
               "ipttt_ff_desc": K.FFDesc, "ipttt_ff_grads": K.FFGrads}
    src = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void){"]
    want = []
    for c, py in structs.items():
        src.append(f'printf("%zu\\n", sizeof({c}));')
        want.append(ctypes.sizeof(py))
        for f, _ in py._fields_:
            src.append(f'printf("%zu\\n", offsetof({c}, {f}));')
            want.append(getattr(py, f).offset)
    (tmp_path / "l.c").write_text("\n".join(src + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == want
    # the binding's flat form of the recurrence has the same fields in the same places
    flat = K._FlatRecurrence
    assert ctypes.sizeof(flat) == ctypes.sizeof(K.RecurrenceDesc)
    for v in "gvh":
        at = getattr(K.RecurrenceDesc, v).offset
        for f, full in (("p", "p"), ("seq", "seq_stride"), ("tok", "tok_stride")):
            assert getattr(flat, f"{v}_{f}").offset == at + getattr(K.View, full).offset
    for f in ("batch", "d", "seq_len", "dtype", "starts", "lens", "h0"):
        assert getattr(flat, f).offset == getattr(K.RecurrenceDesc, f).offset


class FakeMem:
    def __init__(self):
        self.bufs = []

    def ptr(self, offset=0):
        b = ctypes.create_string_buffer(1024)
        self.bufs.append(b)
        return (ctypes.addressof(b) + 255) // 256 * 256 + offset


def refused(status, call, *args, text=None):
    with pytest.raises(B.IptttError) as ei:
        call(*args)
    assert ei.value.status == status, str(ei.value)
    assert str(ei.value).startswith(B.ipttt_status_str(status))
    if text:
        assert text in str(ei.value)


INV, UNS, WSP = B.IPTTT_E_INVALID, B.IPTTT_E_UNSUPPORTED, B.IPTTT_E_WORKSPACE


def test_norm_refusals(lib):
    m = FakeMem()
    p = m.ptr

    def desc(**kw):
        d = dict(d=64, dtype=B.IPTTT_BF16, eps=1e-5, gamma=p(), beta=p())
        d.update(kw)
        return K.NormDesc(**d)

    def fwd(d=None, x=1, xs=64, r=None, rs=0, n=2, h=None, y=1, mean=1, rstd=1):
        v = lambda t: p() if t == 1 else t  # noqa: E731
        K.ipttt_norm_forward(d or desc(), v(x), xs, v(r), rs, n, v(h), v(y), v(mean), v(rstd), 0)

    for kw, status in ((dict(d=0), INV), (dict(d=16385), UNS), (dict(dtype=2), UNS),
                       (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
                       (dict(eps=float("inf")), INV), (dict(gamma=p(1)), INV), (dict(beta=p(1)), INV)):
        refused(status, fwd, desc(**kw))
    for kw in (dict(n=-1), dict(x=None), dict(y=None), dict(x=p(1)), dict(xs=63), dict(r=1, rs=64),
               dict(h=1), dict(r=1, rs=63, h=1), dict(mean=None), dict(rstd=p(2))):
        refused(INV, lambda: fwd(**kw))
    refused(UNS, lambda: fwd(n=1 << 31))
    refused(INV, lambda: fwd(xs=1 << 62), text="too large")
    fwd(n=0, x=None, y=None)   # no rows: nothing to do
    with pytest.raises(B.IptttError):
        B._check(lib.ipttt_norm_forward(None, None, 0, None, 0, 1, None, None, None, None, None))

    ws, need = p(), K.ipttt_norm_backward_workspace_bytes(desc(), 2)
    assert need > 0 and K.ipttt_norm_backward_workspace_bytes(desc(d=0), 2) == 0
    assert K.ipttt_norm_backward_workspace_bytes(desc(), -1) == 0

    def bwd(h=1, hs=64, mean=1, rstd=1, dy=1, ds=64, dh=1, dhs=64, n=2, dx=1, dg=1, db=1, w=ws, wb=need):
        v = lambda t: p() if t == 1 else t  # noqa: E731
        K.ipttt_norm_backward(desc(), v(h), hs, v(mean), v(rstd), v(dy), ds, v(dh), dhs, n, v(dx), v(dg),
                              v(db), w, wb, 0)

    for kw in (dict(h=None), dict(mean=None), dict(rstd=None), dict(dy=None), dict(dx=None),
               dict(dh=p(1)), dict(hs=1), dict(ds=1), dict(dhs=1), dict(dg=p(2)), dict(db=p(1)),
               dict(w=None), dict(w=ws + 64), dict(n=-3)):
        refused(INV, lambda: bwd(**kw))
    refused(WSP, lambda: bwd(wb=need - 1))
    bwd(n=0, dg=None, db=None, w=None, wb=0)


def test_recurrence_refusals(lib):
    m = FakeMem()
    p = m.ptr

    def view(ptr=1, seq=640, tok=64):
        return K.View(p() if ptr == 1 else ptr, seq, tok)

    def rec(**kw):
        d = dict(batch=2, d=64, seq_len=10, dtype=B.IPTTT_BF16, g=view(), v=view(), h=view(),
                 starts=p(), lens=p(), h0=p())
        d.update(kw)
        return K.RecurrenceDesc(**d)

    ws = p()

    def fwd(r=None, last=None, w=ws, wb=None):
        r = r or rec()
        need = K.ipttt_recurrence_workspace_bytes(r)
        K.ipttt_recurrence_forward(r, last, w, need if wb is None else wb, 0)

    bad = [(dict(batch=-1), INV), (dict(batch=1 << 16), UNS), (dict(d=0), INV), (dict(d=65537), UNS),
           (dict(seq_len=-1), INV), (dict(seq_len=(1 << 30) + 1), UNS), (dict(dtype=3), UNS),
           (dict(batch=65535, seq_len=1 << 29, d=65536), UNS),
           (dict(g=view(None)), INV), (dict(v=view(p(1))), INV), (dict(h=view(None)), INV),
           (dict(g=view(tok=63)), INV), (dict(v=view(seq=63)), INV), (dict(h=view(tok=1 << 62)), INV),
           (dict(lens=p(2)), INV), (dict(h0=p(2)), INV)]
    for kw, status in bad:
        refused(status, lambda: fwd(rec(**kw)))
        if not any(isinstance(v, K.View) and v.tok_stride != 64 for v in kw.values()):  # one token: no stride
            refused(status, lambda: K.ipttt_recurrence_step(rec(**{"seq_len": 1, **kw}), p(), 0))
    r = rec()
    refused(INV, lambda: fwd(r, last=r.h0), text="h_last")
    refused(INV, lambda: fwd(last=p(1)))
    refused(INV, lambda: fwd(w=None))
    refused(INV, lambda: fwd(w=ws + 8))
    refused(WSP, lambda: fwd(wb=1))
    refused(INV, lambda: K.ipttt_recurrence_step(rec(), p(), 0), text="seq_len")
    refused(INV, lambda: K.ipttt_recurrence_step(rec(seq_len=1), None, 0))
    fwd(rec(batch=0, g=view(None)))   # no sequence: nothing to do
    assert lib.ipttt_recurrence_forward(None, None, None, 0, None) == INV

    def bwd(r=None, dh=1, dlast=None, dg=1, dv=1, dh0=None, w=ws, wb=None):
        r = r or rec()
        v = lambda t: view() if t == 1 else t  # noqa: E731
        need = K.ipttt_recurrence_workspace_bytes(r)
        K.ipttt_recurrence_backward(r, v(dh), dlast, v(dg), v(dv), dh0, w, need if wb is None else wb, 0)

    for kw in (dict(dh=None), dict(dg=None), dict(dv=None), dict(dh=view(None)), dict(dg=view(tok=1)),
               dict(dv=view(p(1))), dict(dlast=p(2)), dict(dh0=p(2)), dict(w=None)):
        refused(INV, lambda: bwd(**kw))
    refused(INV, lambda: bwd(r, dh0=r.h0), text="dh0")
    same = p()
    refused(INV, lambda: bwd(dlast=same, dh0=same), text="dh0")
    refused(WSP, lambda: bwd(wb=0))


@pytest.mark.parametrize("n,length,d", [(1, 17, 1), (1, 128, 128), (1, 129, 128), (3, 1000, 130),
                                        (2, 131072, 2560), (5, 4097, 33)])
def test_recurrence_workspace_holds_every_tile(lib, n, length, d):
    """Tiles of 128 tokens x 128 channels hand 8 bytes a channel to the tiles behind them."""
    for dtype in (B.IPTTT_F32, B.IPTTT_BF16):
        got = K.ipttt_recurrence_workspace_bytes(K.RecurrenceDesc(batch=n, d=d, seq_len=length, dtype=dtype))
        tiles = -(-length // 128)
        assert got >= 256 + (8 * tiles * n * (-(-d // 128) * 128) if tiles > 1 else 0)


def test_ff_refusals(lib):
    m = FakeMem()
    p = m.ptr

    def desc(**kw):
        d = dict(d=64, d_ff=128, dtype=B.IPTTT_BF16, w_gate=p(), w_up=p(), w_down=p())
        d.update(kw)
        return K.FFDesc(**d)

    ws, need = p(), K.ipttt_ff_workspace_bytes(desc(), 100)
    assert need > 0
    for kw in (dict(d=0), dict(d_ff=0), dict(d=65537), dict(d_ff=262145), dict(dtype=5)):
        assert K.ipttt_ff_workspace_bytes(desc(**kw), 100) == 0
        assert K.ipttt_ff_backward_workspace_bytes(desc(**kw), 100) == 0
    assert K.ipttt_ff_workspace_bytes(desc(), -1) == 0

    def fwd(d=None, x=1, xs=64, n=100, y=1, ys=64, a=None, u=None, w=ws, wb=need):
        v = lambda t: p() if t == 1 else t  # noqa: E731
        K.ipttt_ff_forward(d or desc(), v(x), xs, n, v(y), ys, v(a), v(u), w, wb, 0)

    for kw, status in ((dict(d=0), INV), (dict(d_ff=-1), INV), (dict(d=65537), UNS),
                       (dict(d_ff=1 << 19), UNS), (dict(dtype=7), UNS), (dict(w_gate=None), INV),
                       (dict(w_up=p(8)), INV), (dict(w_down=p(2)), INV)):
        refused(status, lambda: fwd(desc(**kw)))
    for kw in (dict(x=None), dict(y=None), dict(x=p(1)), dict(xs=63), dict(ys=0), dict(a=1), dict(u=1),
               dict(a=p(8), u=1), dict(w=None), dict(w=ws + 16), dict(n=-1)):
        refused(INV, lambda: fwd(**kw))
    refused(UNS, lambda: fwd(n=(1 << 24) + 1))
    refused(WSP, lambda: fwd(wb=need - 1))
    fwd(n=0, x=None, y=None, w=None, wb=0)
    assert lib.ipttt_ff_forward(None, None, 0, 1, None, 0, None, None, None, 0, None) == INV

    bneed = K.ipttt_ff_backward_workspace_bytes(desc(), 100)

    def bwd(x=1, xs=64, a=1, u=1, dy=1, ds=64, n=100, w=ws, wb=bneed, g=1, **kw):
        v = lambda t: p() if t == 1 else t  # noqa: E731
        grads = dict(dx=p(), dx_stride=64, dw_gate=p(), dw_up=p(), dw_down=p())
        grads.update(kw)
        K.ipttt_ff_backward(desc(), v(x), xs, v(a), v(u), v(dy), ds, n, K.FFGrads(**grads) if g else None, w,
                            wb, 0)

    for kw in (dict(x=None), dict(a=None), dict(u=p(4)), dict(dy=None), dict(dy=p(1)), dict(xs=1),
               dict(ds=1), dict(g=None), dict(dx=None), dict(dx_stride=5), dict(dw_gate=None),
               dict(dw_up=p(4)), dict(dw_down=None), dict(w=None), dict(n=-1)):
        refused(INV, lambda: bwd(**kw))
    refused(WSP, lambda: bwd(wb=bneed - 1))


def test_tensor_refusals_on_the_host():
    """What the Python operators refuse before the library is asked: CPU tensors, shapes,
    types, layouts."""
    gamma = torch.ones(8)
    op = K.Norm(gamma)
    refused(INV, op.forward, torch.ones(2, 8), text="not on a GPU")
    refused(INV, op.forward, torch.ones(2, 7))
    refused(INV, op.forward, torch.ones(2, 8, dtype=torch.bfloat16))
    refused(INV, op.forward, torch.ones(8, 2).t())
    refused(UNS, K.Norm, torch.ones(8, dtype=torch.float16))
    refused(INV, K.Norm, gamma, torch.ones(9))
    refused(INV, K.recurrence_forward, torch.ones(2, 3), torch.ones(2, 3))
    refused(INV, K.recurrence_forward, torch.ones(1, 2, 3), torch.ones(1, 2, 3), text="not on a GPU")
    refused(INV, K.recurrence_step, torch.ones(1, 2, 3), torch.ones(1, 2, 3), None)
    w = torch.ones(6, 4)
    refused(INV, K.FeedForward, w, w, w)
    refused(INV, K.FeedForward, torch.ones(4, 6).t(), w, torch.ones(4, 6))
    refused(INV, K.FeedForward(w, w, torch.ones(4, 6)).forward, torch.ones(3, 4), text="not on a GPU")
    # leading dimensions that are not equally spaced rows
    odd = torch.ones(3, 5, 8)[:, :2]
    refused(INV, op.forward, odd, text="equally spaced")


def test_refusals_under_asan(tmp_path):
    """block.cpp and ipttt.cpp under AddressSanitizer and UndefinedBehaviorSanitizer,
    linked with the regular kernel objects, driven by tests/block_abi_asan.c."""
    if not os.path.exists(os.path.join(LLVM, "clang++")):
        pytest.skip("ROCm clang not found")
    objs = [bld.object_path(s) for s in bld.SOURCES if s.endswith(".hip")]
    missing = [o for o in objs if not os.path.exists(o)]
    if missing:
        pytest.fail(f"kernel objects missing ({missing[0]}): run __graft_entry__.build()")
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer",
           "-g", "-Wall", "-Wextra", "-Werror"]

    def run(cmd, **kw):
        r = subprocess.run(cmd, capture_output=True, text=True, **kw)
        assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
        return r

    for src in ("ipttt.cpp", "block.cpp"):
        objs.append(str(tmp_path / (src + ".o")))
        run([f"{LLVM}/clang++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", *san, "-c",
             os.path.join(ROOT, "chunked_weight_mlp_amd", "csrc", src), "-o", objs[-1]])
    main = str(tmp_path / "main.o")
    run([f"{LLVM}/clang", "-std=c99", *san, "-I", os.path.join(ROOT, "include"), "-c",
         os.path.join(ROOT, "tests", "block_abi_asan.c"), "-o", main])
    exe = str(tmp_path / "block_abi_asan")
    run([f"{LLVM}/clang++", "-fsanitize=address,undefined", main, *objs, "-L/opt/rocm/lib", "-lamdhip64",
         "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    r = run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
                            UBSAN_OPTIONS="print_stacktrace=1"), timeout=120)
    assert "all checks passed" in r.stdout


def test_widths_of_zero_are_refused():
    """An operator over no columns: an error of the library's kind, not of arithmetic."""
    refused(INV, K.Norm, torch.ones(0), text="d > 0")
    for f, d in ((0, 4), (6, 0), (0, 0)):
        refused(INV, K.FeedForward, torch.ones(f, d), torch.ones(f, d), torch.ones(d, f), text="> 0")


@pytest.mark.parametrize("n,length,d", [(1, 1025, 128), (1, 9000, 130), (3, 1000, 130), (2, 131072, 2560),
                                        (5, 4097, 33), (2, 20000, 64)])
def test_recurrence_workspace_holds_the_groups_of_tiles(lib, n, length, d):
    """Behind the tiles' slots lie those of their groups, of 8 tiles each and one begun."""
    for dtype in (B.IPTTT_F32, B.IPTTT_BF16):
        got = K.ipttt_recurrence_workspace_bytes(K.RecurrenceDesc(batch=n, d=d, seq_len=length, dtype=dtype))
        tiles = -(-length // 128)
        width = -(-d // 128) * 128 if d > 64 else 64
        assert got >= 256 + 8 * (tiles + tiles // 8 + 1) * n * width


@pytest.mark.parametrize("dtype", [B.IPTTT_F32, B.IPTTT_BF16])
@pytest.mark.parametrize("d,f", [(1024, 4096), (2048, 8192), (2560, 9728), (4096, 16384)])
def test_few_tokens_backward_lays_out_no_weights(lib, d, f, dtype):
    """To 320 tokens of any size the products take the weights as they lie, which is the
    faster of the two ways there: the workspace holds no copies of them."""
    desc, e = K.FFDesc(d=d, d_ff=f, dtype=dtype), 2 if dtype == B.IPTTT_BF16 else 4
    for n in (1, 64, 129, 193, 256, 320):
        z, sums = 3 * n * f * e, 64 * 4 * n * (d + 8)   # dA, dU, z; dx's partial sums
        assert K.ipttt_ff_backward_workspace_bytes(desc, n) <= z + sums + 4096
    # and with very many they are copied (bf16) or split into planes (fp32)
    assert K.ipttt_ff_backward_workspace_bytes(desc, 1 << 15) >= 3 * d * f * (2 if e == 2 else 6)
