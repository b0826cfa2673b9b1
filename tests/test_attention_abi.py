"""C-ABI checks of include/ipttt_attention.h that need no GPU: exports, structure layouts,
workspace sizes, and every refusal, before any device work (the pointers are host memory)."""
from __future__ import annotations

import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

from chunked_weight_mlp_amd import attention as A
from chunked_weight_mlp_amd import build as bld
from chunked_weight_mlp_amd import ipttt as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ipttt_attention.h")
LLVM = "/opt/rocm/llvm/bin"
INV, UNS, WSP = B.IPTTT_E_INVALID, B.IPTTT_E_UNSUPPORTED, B.IPTTT_E_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.fail("libipttt.so is not built: run __graft_entry__.build()")
    return A.load()


def test_header_declares_the_binding_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(ipttt_[a-z_]+)\s*\(", text))) == sorted(A.EXPORTS)
    for f in A.EXPORTS:
        assert hasattr(lib, f)


def test_structure_layouts_match_c(tmp_path):
    structs = {"ipttt_heads": A.Heads, "ipttt_kv_cache": A.KVCacheDesc, "ipttt_page_table": A.PageTable,
               "ipttt_headnorm_desc": A.HeadNormDesc, "ipttt_attention": A.AttentionDesc,
               "ipttt_step_desc": A.StepDesc}
    src = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void){"]
    want = []
    for c, py in structs.items():
        src.append(f'printf("%zu\\n", sizeof({c}));')
        want.append(ctypes.sizeof(py))
        for f, _ in py._fields_:
            src.append(f'printf("%zu\\n", offsetof({c}, {f}));')
            want.append(getattr(py, f).offset)
    (tmp_path / "l.c").write_text("\n".join(src + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(tmp_path / "l.c"), "-o", str(tmp_path / "l")],
                   check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == want


class Mem:
    def __init__(self):
        self.bufs = []

    def __call__(self, offset=0):
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


def test_headnorm_refusals(lib):
    p = Mem()

    def desc(**kw):
        d = dict(q_heads=2, k_heads=1, head_dim=64, rotary=32, interleaved=0, dtype=B.IPTTT_BF16, eps=1e-6,
                 q_gamma=p(), k_gamma=p(), inv_freq=p())
        d.update(kw)
        return A.HeadNormDesc(**d)

    def heads(ptr=1, tok=128, head=64):
        return A.Heads(p() if ptr == 1 else ptr, tok, head)

    def fwd(d=None, n=2, pos=1, **kw):
        v = dict(q=heads(), k=heads(), q_out=heads(), k_out=heads())
        v.update(kw)
        A.ipttt_headnorm_forward(d or desc(), v["q"], v["k"], p() if pos == 1 else pos, n, v["q_out"], v["k_out"], 0)

    bad = [(dict(q_heads=0), INV), (dict(k_heads=-1), INV), (dict(q_heads=1025), UNS), (dict(head_dim=0), INV),
           (dict(head_dim=129), UNS), (dict(rotary=3), INV), (dict(rotary=66), INV), (dict(rotary=-2), INV),
           (dict(dtype=2), UNS), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(eps=math.inf), INV),
           (dict(q_gamma=p(1)), INV), (dict(k_gamma=p(1)), INV), (dict(inv_freq=None), INV),
           (dict(inv_freq=p(4)), INV)]
    for kw, status in bad:
        refused(status, fwd, desc(**kw))
    for name in ("q", "k", "q_out", "k_out"):
        for h in (None, heads(None), heads(p(1)), heads(tok=63), heads(tok=1 << 62)):
            refused(INV, lambda: fwd(**{name: h}))
    for name in ("q", "q_out"):
        refused(INV, lambda: fwd(**{name: heads(head=63)}), text="head stride")
    refused(INV, lambda: fwd(n=-1))
    refused(UNS, lambda: fwd(n=1 << 31))
    refused(INV, lambda: fwd(pos=None))
    refused(INV, lambda: fwd(pos=p(2)))
    fwd(n=0, q=heads(None), k=heads(None), q_out=heads(None), k_out=heads(None), pos=None)

    cache = dict(k=p(), v=p(), pages=4, page_size=16, k_heads=1, head_dim=64, dtype=B.IPTTT_BF16)
    tab = dict(p=p(), stride=4, batch=2, width=4)

    def app(n=2, pos=1, seqs=None, v=1, ckw=None, tkw=None):
        A.ipttt_headnorm_append(desc(), heads(), heads(), heads() if v == 1 else v, p() if pos == 1 else pos, seqs, n,
                                heads(), A.KVCacheDesc(**{**cache, **(ckw or {})}),
                                A.PageTable(**{**tab, **(tkw or {})}), 0)

    for kw, status in ((dict(k=None), INV), (dict(v=p(8)), INV), (dict(pages=-1), INV), (dict(page_size=0), INV),
                       (dict(page_size=65537), UNS), (dict(k_heads=2), INV), (dict(head_dim=32), INV),
                       (dict(dtype=B.IPTTT_F32), INV), (dict(dtype=9), UNS)):
        refused(status, lambda: app(ckw=kw))
    for kw, status in ((dict(p=None), INV), (dict(p=p(2)), INV), (dict(stride=3), INV), (dict(batch=-1), INV),
                       (dict(batch=65536), UNS), (dict(width=-1), INV), (dict(width=1 << 28), UNS)):
        refused(status, lambda: app(tkw=kw))
    refused(INV, lambda: app(v=heads(None)))
    refused(INV, lambda: app(seqs=p(1)))
    refused(INV, lambda: app(pos=None))
    app(n=0)

    need = A.ipttt_headnorm_backward_workspace_bytes(desc(), 2)
    assert need > 0 and A.ipttt_headnorm_backward_workspace_bytes(desc(head_dim=0), 2) == 0
    assert A.ipttt_headnorm_backward_workspace_bytes(desc(), -1) == 0
    ws = p()

    def bwd(d=None, n=2, dg=1, w=ws, wb=need, **kw):
        v = dict(q=heads(), k=heads(), dq=heads(), dk=heads(), ox=heads(), ok=heads())
        v.update(kw)
        g = p() if dg == 1 else dg
        A.ipttt_headnorm_backward(d or desc(), v["q"], v["k"], p(), v["dq"], v["dk"], n, v["ox"], v["ok"], g, g, w, wb, 0)

    for name in ("q", "k", "dq", "dk", "ox", "ok"):
        refused(INV, lambda: bwd(**{name: heads(None)}))
        refused(INV, lambda: bwd(**{name: heads(tok=8)}))
    refused(INV, lambda: bwd(dg=p(2)))
    refused(INV, lambda: bwd(desc(q_gamma=None)), text="gradient")
    refused(INV, lambda: bwd(w=None))
    refused(INV, lambda: bwd(w=ws + 16))
    refused(WSP, lambda: bwd(wb=need - 1))
    bwd(n=0, dg=None, w=None, wb=0)


def test_attention_refusals(lib):
    p = Mem()

    def desc(**kw):
        d = dict(q_heads=4, k_heads=2, head_dim=64, batch=1, causal=1, window=0, dtype=B.IPTTT_BF16, scale=0.125,
                 n_q=2, n_k=3, q_offsets=p(), k_offsets=p())
        d.update(kw)
        return A.AttentionDesc(**d)

    def heads(ptr=1, tok=256, head=64):
        return A.Heads(p() if ptr == 1 else ptr, tok, head)

    ws = p()
    need = A.ipttt_attention_forward_workspace_bytes(desc())
    bneed = A.ipttt_attention_backward_workspace_bytes(desc())
    assert 0 < need <= 1024 and bneed >= need + 4 * 2 * 8

    def fwd(d=None, lse=1, w=ws, wb=1 << 20, **kw):
        v = dict(q=heads(), k=heads(), v=heads(), o=heads())
        v.update(kw)
        A.ipttt_attention_forward(d or desc(), v["q"], v["k"], v["v"], v["o"], p() if lse == 1 else lse, w, wb, 0)

    def bwd(d=None, lse=1, w=ws, wb=1 << 20, **kw):
        v = {x: heads() for x in ("q", "k", "v", "o", "dy", "dq", "dk", "dv")}
        v.update(kw)
        A.ipttt_attention_backward(d or desc(), v["q"], v["k"], v["v"], v["o"], p() if lse == 1 else lse, v["dy"],
                                   v["dq"], v["dk"], v["dv"], w, wb, 0)

    bad = [(dict(q_heads=0), INV), (dict(k_heads=0), INV), (dict(q_heads=5), INV), (dict(q_heads=2048), UNS),
           (dict(head_dim=0), INV), (dict(head_dim=129), UNS), (dict(batch=-1), INV), (dict(batch=65536), UNS),
           (dict(window=-1), INV), (dict(window=4, causal=0), INV), (dict(dtype=4), UNS), (dict(scale=math.nan), INV),
           (dict(scale=math.inf), INV), (dict(n_q=-1), INV), (dict(n_k=-1), INV), (dict(n_q=(1 << 30) + 1), UNS),
           (dict(n_k=(1 << 30) + 1), UNS), (dict(q_heads=1024, n_q=1 << 30), UNS), (dict(q_offsets=None), INV),
           (dict(k_offsets=None), INV), (dict(q_offsets=None, k_offsets=None, batch=2), INV),
           (dict(q_offsets=p(2)), INV), (dict(k_offsets=p(1)), INV)]
    for kw, status in bad:
        refused(status, fwd, desc(**kw))
        refused(status, bwd, desc(**kw))
    for kw in (dict(q_heads=0), dict(head_dim=200), dict(n_q=-1), dict(batch=1 << 20)):
        assert A.ipttt_attention_forward_workspace_bytes(desc(**kw)) == 0
        assert A.ipttt_attention_backward_workspace_bytes(desc(**kw)) == 0
    for call, names in ((fwd, ("q", "k", "v", "o")), (bwd, ("q", "k", "v", "o", "dy", "dq", "dk", "dv"))):
        for name in names:
            for h in (None, heads(None), heads(p(1)), heads(tok=63), heads(head=63), heads(tok=1 << 61),
                      heads(head=1 << 61)):
                refused(INV, lambda: call(**{name: h}))
        refused(INV, lambda: call(lse=p(2)))
        refused(INV, lambda: call(w=None))
        refused(INV, lambda: call(w=ws + 4))
    refused(INV, lambda: bwd(lse=None))
    refused(WSP, lambda: fwd(wb=need - 1))
    refused(WSP, lambda: bwd(wb=bneed - 1))
    z = heads(None)
    fwd(desc(n_q=0, n_k=0), lse=None, w=None, wb=0, q=z, k=z, v=z, o=z)
    bwd(desc(n_q=0, n_k=0), lse=None, w=None, wb=0, q=z, k=z, v=z, o=z, dy=z, dq=z, dk=z, dv=z)


def test_step_refusals(lib):
    p = Mem()
    cache = dict(k=p(), v=p(), pages=4, page_size=16, k_heads=2, head_dim=64, dtype=B.IPTTT_F32)
    tab = dict(p=p(), stride=64, batch=2, width=64)
    ws = p()

    def step(dkw=None, ckw=None, tkw=None, q=1, o=1, lens=1, lse=None, w=ws, wb=1 << 30):
        hd = lambda t: A.Heads(p(), 256, 64) if t == 1 else t  # noqa: E731
        A.ipttt_attention_step(A.StepDesc(**{**dict(q_heads=4, window=0, scale=0.1), **(dkw or {})}), hd(q),
                               A.KVCacheDesc(**{**cache, **(ckw or {})}), A.PageTable(**{**tab, **(tkw or {})}),
                               p() if lens == 1 else lens, hd(o), lse, w, wb, 0)

    for kw, status in ((dict(q_heads=0), INV), (dict(q_heads=3), INV), (dict(q_heads=1026), UNS),
                       (dict(window=-1), INV), (dict(scale=math.inf), INV)):
        refused(status, lambda: step(dkw=kw))
    for kw, status in ((dict(k=None), INV), (dict(v=p(4)), INV), (dict(pages=-1), INV), (dict(page_size=0), INV),
                       (dict(page_size=1 << 20), UNS), (dict(k_heads=0), INV), (dict(head_dim=129), UNS),
                       (dict(dtype=3), UNS)):
        refused(status, lambda: step(ckw=kw))
    for kw, status in ((dict(p=None), INV), (dict(p=p(1)), INV), (dict(stride=63), INV), (dict(batch=-1), INV),
                       (dict(batch=70000), UNS), (dict(width=-2), INV), (dict(width=1 << 27), UNS)):
        refused(status, lambda: step(tkw=kw))
    for kw in (dict(q=None), dict(o=None), dict(q=A.Heads(None, 256, 64)), dict(o=A.Heads(p(2), 256, 64)),
               dict(q=A.Heads(p(), 32, 64)), dict(lens=None), dict(lens=p(2)), dict(lse=p(2)), dict(w=None),
               dict(w=ws + 128)):
        refused(INV, lambda: step(**kw))
    args = (A.StepDesc(4, 0, 0.1), A.KVCacheDesc(**cache), A.PageTable(**tab))
    need = A.ipttt_attention_step_workspace_bytes(*args)
    assert need > 0
    refused(WSP, lambda: step(wb=need - 1))
    assert A.ipttt_attention_step_workspace_bytes(A.StepDesc(3, 0, 0.1), *args[1:]) == 0
    assert A.ipttt_attention_step_workspace_bytes(args[0], A.KVCacheDesc(**{**cache, "page_size": 0}), args[2]) == 0
    assert A.ipttt_attention_step_workspace_bytes(*args[:2], A.PageTable(**{**tab, "batch": -1})) == 0
    # short tables are not split and need no more than the minimum
    assert A.ipttt_attention_step_workspace_bytes(*args[:2], A.PageTable(**{**tab, "width": 4})) == 256
    step(tkw=dict(batch=0), q=A.Heads(None, 0, 0), o=A.Heads(None, 0, 0), lens=None, w=None, wb=0)


def test_tensor_refusals_on_the_host():
    """What the Python operators refuse before the library is asked."""
    f = torch.ones(8, dtype=torch.float64)
    g = torch.ones(16)
    refused(INV, A.HeadNorm, g[:0], None, f, text="head_dim > 0")
    refused(INV, A.HeadNorm, None, None, f, text="must be given")
    refused(INV, A.HeadNorm, g, torch.ones(15), f)
    refused(INV, A.HeadNorm, g, g.to(torch.bfloat16), f)
    refused(UNS, A.HeadNorm, g.half(), None, f)
    refused(UNS, lambda: A.HeadNorm(None, None, f, head_dim=16, dtype=torch.float16))
    refused(INV, A.HeadNorm, g, g, torch.ones(8, dtype=torch.int64))
    op = A.HeadNorm(g, g, f)
    q, k, pos = torch.ones(3, 2, 16), torch.ones(3, 1, 16), torch.zeros(3, dtype=torch.int32)
    refused(INV, op.forward, q, k, pos, text="not on a GPU")
    refused(INV, op.forward, q[0], k, pos)
    refused(INV, op.forward, q[..., :15], k, pos)
    refused(INV, op.forward, q, k[:2], pos)
    refused(INV, op.forward, q.bfloat16(), k, pos)
    refused(INV, op.forward, q, k, pos.long())
    refused(INV, op.forward, q, k, pos[:2])
    refused(INV, op.forward, torch.ones(3, 16, 2).transpose(1, 2), k, pos, text="channels")
    refused(INV, op.backward, q, k, pos, q[:, :1], k)
    pages = torch.ones(4, 1, 8, 16)
    refused(INV, A.KVCache, pages[0], pages[0])
    refused(INV, A.KVCache, pages, pages[:3])
    two = torch.ones(4, 2, 8, 16).transpose(1, 2)
    refused(INV, A.KVCache, two, two, text="contiguous")
    refused(UNS, A.KVCache, pages.double(), pages.double())
    cache, table, lens = A.KVCache(pages, pages), torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    refused(INV, op.append, q, k, k, pos, cache, table, text="not on a GPU")
    refused(INV, op.append, q, k, q, pos, cache, table)
    refused(INV, op.append, q, k, k, pos, cache, table.long())
    refused(INV, op.append, q, k, k, pos, cache, table[0])
    refused(INV, op.append, q, k, k, pos, cache, table, pos.long())
    refused(INV, A.attention_step, q, cache, table, lens, text="not on a GPU")
    refused(INV, A.attention_step, q[:2], cache, table, lens[:2])
    refused(INV, A.attention_step, q, cache, table, lens.long())
    refused(INV, A.attention_step, q.bfloat16(), cache, table, lens)
    refused(INV, A.attention_step, q, cache, torch.zeros(2, 3, dtype=torch.int32).t(), lens, text="rows contiguous")
    off = torch.zeros(2, dtype=torch.int32)
    refused(INV, A.attention_forward, q, k, k, text="not on a GPU")
    refused(INV, A.attention_forward, q, k, k[:2])
    refused(INV, A.attention_forward, q, k[:2], k[:2], off, text="k_offsets")
    refused(INV, A.attention_forward, q, k, k, None, off, text="without offsets")
    refused(INV, A.attention_forward, q, k, k, off, off[:1])
    refused(INV, A.attention_forward, q, k, k, off[:0], off[:0])
    refused(INV, A.attention_forward, q, k, k, off.long())
    refused(UNS, A.attention_forward, q.half(), k.half(), k.half())
    for w in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1):
        refused(INV, lambda: A.attention_forward(q, k, k, window=w), text="32 bits")
    refused(INV, A.attention_backward, q, k, k, q, torch.ones(3, 2), q, text="lse")
    refused(INV, A.attention_backward, q, k, k, q[:2], torch.ones(2, 3), q)


def test_refusals_under_asan(tmp_path):
    """attention.cpp and ipttt.cpp under AddressSanitizer and UndefinedBehaviorSanitizer, linked
    with the regular kernel objects, driven by tests/attention_abi_asan.c."""
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

    for src in ("ipttt.cpp", "attention.cpp"):
        objs.append(str(tmp_path / (src + ".o")))
        run([f"{LLVM}/clang++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", *san, "-c",
             os.path.join(ROOT, "chunked_weight_mlp_amd", "csrc", src), "-o", objs[-1]])
    main = str(tmp_path / "main.o")
    run([f"{LLVM}/clang", "-std=c99", *san, "-I", os.path.join(ROOT, "include"), "-c",
         os.path.join(ROOT, "tests", "attention_abi_asan.c"), "-o", main])
    exe = str(tmp_path / "attention_abi_asan")
    run([f"{LLVM}/clang++", "-fsanitize=address,undefined", main, *objs, "-L/opt/rocm/lib", "-lamdhip64",
         "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    r = run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
                            UBSAN_OPTIONS="print_stacktrace=1"), timeout=120)
    assert "all checks passed" in r.stdout
