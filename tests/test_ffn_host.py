"""The feed-forward library on the host: it loads, exports what
include/tgemm_ffn.h declares, its argument structs are those of the binding,
and bad arguments are refused with the documented status before any device is
touched.  No test here launches a kernel."""
import os
import re
import subprocess

import pytest
import torch

import dense_tiled_gemm_bf16_amd as tg
from dense_tiled_gemm_bf16_amd import ffn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tgemm_ffn.h")

# Plausible device addresses, 64 GiB apart; a refused call uses none.
P = [0x10000 + (i << 36) for i in range(1, 12)]


def call(name, **fields):
    return getattr(ffn.lib(), name)(ffn.args(name, **fields), None)


def refused(name, code, word, **fields):
    rc = call(name, **fields)
    assert rc == code, (rc, ffn.last_error())
    assert word in ffn.last_error(), ffn.last_error()


def test_exports_what_the_header_declares():
    declared = set(re.findall(r"^TGEMM_API\s+[\w\s\*]*?\b(\w+)\s*\(", open(HEADER).read(), re.M))
    ffn.lib()
    out = subprocess.run(["nm", "-D", "--defined-only", ffn.LIB_PATH], capture_output=True, text=True, check=True)
    assert {l.split()[-1] for l in out.stdout.splitlines() if " T " in l} == declared


def test_header_compiles_as_c_and_structs_match():
    text = open(HEADER).read()
    structs = dict((name, body) for body, name in re.findall(r"typedef struct \{(.*?)\} (\w+);", text, re.S))
    by_call = dict(re.findall(r"TGEMM_API int (\w+)\(const (\w+) \*args", text))
    assert set(by_call) == set(ffn._FIELDS)
    checks = ""
    for call_name, struct_name in by_call.items():
        fields = []
        for decl in structs[struct_name].split(";"):
            decl = decl.strip()
            if decl:
                fields += [re.sub(r".*[\s\*]", "", part.strip()) for part in decl.split(",")]
        assert fields == ffn._FIELDS[call_name].split(), call_name
        checks += f"_Static_assert(sizeof({struct_name}) == {8 * len(fields)}, \"{struct_name}\");\n"
        assert len(ffn.args(call_name)) == 8 * len(fields)
    src = '#include "tgemm_ffn.h"\n' + checks + "int main(void){ return TGEMM_OK; }\n"
    res = subprocess.run(["gcc", "-x", "c", "-std=c11", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                          "-I", "/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-"], input=src, text=True,
                         capture_output=True)
    assert res.returncode == 0, res.stderr


def epi(**kw):
    base = dict(dtype=0, trans_b=1, M=16, N=32, K=64, A=P[0], lda=64, B=P[1], ldb=64, C=P[2], ldc=32)
    base.update(kw)
    return base


def deep(**kw):
    """A call whose K is split."""
    return epi(K=8192, lda=8192, ldb=8192, workspace_bytes=1 << 20, **kw)


@pytest.mark.parametrize("fields,code,word", [
    (epi(dtype=2), tg.EINVAL, "element type"), (epi(trans_a=2), tg.EINVAL, "trans_a"),
    (epi(M=-1), tg.EINVAL, "negative"), (epi(M=1 << 31), tg.ETOOBIG, "below 2^31"),
    (epi(act=7), tg.EINVAL, "activation"), (epi(act=-1), tg.EINVAL, "activation"),
    (epi(act=5, N=24, ldc=16), tg.EALIGN, "multiple of 16"), (epi(act=5, trans_a=1), tg.EINVAL, "gated"),
    (epi(A=0), tg.EINVAL, "A is NULL"), (epi(C=0), tg.EINVAL, "C is NULL"), (epi(B=P[1] + 8), tg.EALIGN, "B is not"),
    (epi(lda=56), tg.EINVAL, "stride of A"), (epi(lda=68), tg.EALIGN, "stride of A"),
    (epi(K=60, lda=64, ldb=64), tg.EALIGN, "row length of A"), (epi(N=36, ldc=40), tg.EALIGN, "row length of C"),
    (epi(ldc=24), tg.EINVAL, "stride of C"), (epi(bias=P[3] + 2), tg.EALIGN, "bias"),
    (epi(residual=P[4], ldr=24), tg.EINVAL, "stride of residual"),
    (epi(preact=P[5], ldp=16), tg.EINVAL, "stride of preact"),
    (epi(C=P[0]), tg.EINVAL, "C overlaps A"), (epi(preact=P[2], ldp=32), tg.EINVAL, "overlaps"),
    (epi(residual=P[2], ldr=40), tg.EINVAL, "C overlaps residual"),
    (epi(residual=P[2] + 16, ldr=32), tg.EINVAL, "C overlaps residual"),
    (epi(preact=P[5], ldp=32, residual=P[5], ldr=32), tg.EINVAL, "preact overlaps residual"),
    (epi(lda=1 << 23, ldb=64), tg.ETOOBIG, "A too large"), (epi(ldb=1 << 23), tg.ETOOBIG, "B too large"),
    (epi(act=5, N=1 << 22, ldb=512, ldc=1 << 21), tg.ETOOBIG, "B too large"),
    (epi(lda=1 << 31), tg.ETOOBIG, "stride of A"),
    (deep(workspace=P[3] + 4), tg.EALIGN, "workspace"), (deep(workspace=P[0] + 4096), tg.EINVAL, "workspace overlaps A"),
    (deep(workspace=P[2]), tg.EINVAL, "C overlaps workspace"),
    (deep(workspace=P[4] + 64, residual=P[4], ldr=32), tg.EINVAL, "workspace overlaps residual"),
])
def test_epilogue_refuses(fields, code, word):
    refused("gemm_epilogue", code, word, **fields)


def test_null_argument_structs_are_refused():
    for name in ffn._FIELDS:
        assert getattr(ffn.lib(), name)(None, None) == tg.EINVAL
        assert "args is NULL" in ffn.last_error()


def test_nothing_to_do_needs_no_device():
    assert call("gemm_epilogue", **epi(M=0, A=0, C=0)) == tg.OK
    assert call("gemm_epilogue", **deep(M=0, A=0, C=0, workspace=P[3])) == tg.OK
    assert call("gemm_grouped", dtype=0, trans_b=1, R=0, N=32, K=64, groups=4) == tg.OK
    assert call("gemm_grouped", dtype=0, trans_b=1, R=8, N=32, K=64, groups=0) == tg.OK
    assert call("gemm_grouped_tn", dtype=0, R=8, P=0, Q=8, groups=2) == tg.OK
    assert call("gemm_epilogue_backward", dtype=0, M=0, N=32, act=1) == tg.OK
    assert call("route_topk", dtype=2, T=0, E=8, k=2, groups=1, groups_used=1, scale=1.0) == tg.OK
    assert call("route_topk_backward", dtype=2, T=0, E=8, k=2, scale=1.0) == tg.OK
    assert call("expert_gather", R=0, D=8, src_rows=1) == tg.OK
    assert call("expert_combine", dtype=0, T=0, D=8, R=1, k=1) == tg.OK
    assert call("expert_combine_backward", dtype=0, T=0, D=8, R=1, k=1) == tg.OK


def bwd(**kw):
    base = dict(dtype=0, M=128, N=64, dout=P[0], ldd=64, preact=P[1], ldp=64, act=4, dz=P[2], ldz=64, dbias=P[3],
                workspace=P[4], workspace_bytes=1 << 20)
    base.update(kw)
    return base


@pytest.mark.parametrize("fields,code,word", [
    (bwd(act=9), tg.EINVAL, "activation"), (bwd(dout=0), tg.EINVAL, "dout is NULL"),
    (bwd(preact=0), tg.EINVAL, "preact is NULL"), (bwd(dz=0), tg.EINVAL, "dz is NULL"),
    (bwd(workspace=0), tg.EINVAL, "workspace is NULL"), (bwd(workspace_bytes=16), tg.EINVAL, "workspace bytes"),
    (bwd(workspace=P[4] + 4), tg.EALIGN, "workspace"), (bwd(groups=3), tg.EINVAL, "offsets is NULL"),
    (bwd(dz=P[0] + 128), tg.EINVAL, "dz overlaps dout"), (bwd(dbias=P[2]), tg.EINVAL, "overlaps"),
    (bwd(act=5, dz=P[0], ldd=32, dout=P[0]), tg.EINVAL, "dz overlaps dout"),
    (bwd(ldd=32), tg.EINVAL, "stride of dout"), (bwd(groups=-1), tg.EINVAL, "negative"),
])
def test_epilogue_backward_refuses(fields, code, word):
    refused("gemm_epilogue_backward", code, word, **fields)


def grp(**kw):
    base = dict(dtype=0, trans_b=1, R=64, N=32, K=64, groups=4, offsets=P[5], src_rows=64, A=P[0], lda=64, B=P[1],
                ldb=64, stride_b=32 * 64, C=P[2], ldc=32)
    base.update(kw)
    return base


@pytest.mark.parametrize("fields,code,word", [
    (grp(offsets=0), tg.EINVAL, "offsets is NULL"), (grp(offsets=P[5] + 2), tg.EALIGN, "offsets"),
    (grp(rows=P[6] + 1), tg.EALIGN, "rows"), (grp(stride_b=-8), tg.EINVAL, "stride_b"),
    (grp(stride_b=4), tg.EALIGN, "stride_b"), (grp(stride_b=1 << 41), tg.ETOOBIG, "stride_b"),
    (grp(C=P[1] + 3 * 32 * 64 * 2), tg.EINVAL, "C overlaps B"), (grp(act=6, N=40, ldc=24), tg.EALIGN, "multiple of 16"),
    (grp(rows=P[6], src_rows=1 << 25), tg.ETOOBIG, "A too large"), (grp(groups=-1), tg.EINVAL, "negative"),
    (grp(A=0), tg.EINVAL, "A is NULL"), (grp(trans_b=3), tg.EINVAL, "trans_b"),
    (grp(preact=P[7], ldp=8), tg.EINVAL, "stride of preact"), (grp(K=4), tg.EALIGN, "row length of A"),
])
def test_grouped_refuses(fields, code, word):
    refused("gemm_grouped", code, word, **fields)


def tn(**kw):
    base = dict(dtype=0, R=64, P=32, Q=64, groups=4, offsets=P[5], X=P[0], ldx=32, Y=P[1], ldy=64, out=P[2])
    base.update(kw)
    return base


@pytest.mark.parametrize("fields,code,word", [
    (tn(P=36, ldx=40), tg.EALIGN, "multiple of 8"), (tn(Q=60), tg.EALIGN, "multiple of 8"),
    (tn(out=0), tg.EINVAL, "out is NULL"), (tn(out=P[0]), tg.EINVAL, "out overlaps X"),
    (tn(ldx=1 << 26), tg.ETOOBIG, "X too large"), (tn(ldy=1 << 26), tg.ETOOBIG, "Y too large"),
    (tn(groups=1 << 27), tg.ETOOBIG, "groups"), (tn(offsets=0), tg.EINVAL, "offsets"),
])
def test_grouped_tn_refuses(fields, code, word):
    refused("gemm_grouped_tn", code, word, **fields)


def top(**kw):
    base = dict(dtype=2, T=8, E=64, logits=P[0], ld=64, bias=P[1], k=4, score=1, groups=8, groups_used=4,
                renormalize=1, scale=1.0, weights=P[2], ids=P[3])
    base.update(kw)
    return base


@pytest.mark.parametrize("fields,code,word", [
    (top(dtype=3), tg.EINVAL, "element type"), (top(E=1025, ld=1025, groups=1, groups_used=1), tg.EINVAL, "E="),
    (top(E=0), tg.EINVAL, "E="), (top(k=0), tg.EINVAL, "k="), (top(k=65, E=128, ld=128), tg.EINVAL, "k="),
    (top(k=9, E=8, groups=1, groups_used=1), tg.EINVAL, "k="), (top(groups=7), tg.EINVAL, "groups"),
    (top(groups=128, E=128, ld=128), tg.EINVAL, "groups"), (top(groups_used=9), tg.EINVAL, "groups_used"),
    (top(groups_used=0), tg.EINVAL, "groups_used"), (top(k=33), tg.EINVAL, "experts of groups_used"),
    (top(score=2), tg.EINVAL, "score"), (top(renormalize=2), tg.EINVAL, "renormalize"),
    (top(logits=0), tg.EINVAL, "logits"), (top(logits=P[0] + 2), tg.EALIGN, "logits"),
    (top(ld=32), tg.EINVAL, "stride of logits"), (top(ids=P[2]), tg.EINVAL, "overlaps"),
    (top(T=1 << 30), tg.ETOOBIG, "T k"), (top(ld=1 << 26), tg.ETOOBIG, "16 row strides"),
])
def test_route_topk_refuses(fields, code, word):
    refused("route_topk", code, word, **fields)


BIG = (1 << 31) - 4096  # (a multiple of 8)


def test_sizes_leave_room_for_32_bit_indexes():
    """The first size past the limit is refused; the last before it gets to
    the next check."""
    for size in (BIG, (1 << 31) - 8):
        for name, fields in (("gemm_epilogue", epi(M=size)), ("gemm_epilogue", epi(N=size)),
                             ("gemm_epilogue", epi(K=size)), ("gemm_epilogue_backward", bwd(M=size)),
                             ("gemm_epilogue_backward", bwd(N=size)), ("gemm_grouped", grp(R=size)),
                             ("gemm_grouped", grp(rows=P[6], src_rows=size)), ("gemm_grouped_tn", tn(R=size)),
                             ("expert_gather", dict(R=8, D=size, src_rows=8, x=P[0], ldx=64, rows=P[1], out=P[2])),
                             ("expert_combine", dict(dtype=0, T=1, D=8, R=1, k=size)),
                             ("expert_combine_backward", dict(dtype=0, T=1, D=size, R=1, k=1))):
            refused(name, tg.ETOOBIG, "sizes must be", **fields)
    refused("expert_combine", tg.ETOOBIG, "T k", dtype=0, T=2, D=8, R=1, k=BIG // 2)
    refused("expert_gather", tg.EINVAL, "out is NULL", R=8, D=BIG - 8, src_rows=8, x=P[0], ldx=BIG, rows=P[1], out=0)


def test_groups_and_choices_are_limited():
    refused("gemm_grouped", tg.ETOOBIG, "65536", **grp(groups=65537))
    refused("gemm_grouped", tg.EINVAL, "C is NULL", **grp(groups=65536, C=0))
    refused("gemm_grouped_tn", tg.ETOOBIG, "65536", **tn(groups=65537))
    refused("gemm_epilogue_backward", tg.ETOOBIG, "65536", **bwd(groups=65537, offsets=P[5]))
    plan = dict(T=(1 << 26) + 1, k=1, E=8, ids=P[0], offsets=P[1], rows=P[2], slots=P[3], workspace=P[4])
    refused("route_plan", tg.ETOOBIG, "T k", **plan)
    refused("route_plan", tg.EINVAL, "workspace bytes", **{**plan, "T": 1 << 26})
    assert ffn.lib().tgemm_route_plan_workspace_bytes(1 << 26, 1, 8) == (1 << 14) * 8 * 4
    assert ffn.lib().tgemm_route_plan_workspace_bytes((1 << 26) + 1, 1, 8) == 0


def test_other_calls_refuse():
    r = dict(dtype=0, T=8, E=64, logits=P[0], ld=64, ids=P[1], dweights=P[2], k=4, scale=1.0, dlogits=P[3], ldo=64)
    refused("route_topk_backward", tg.EINVAL, "dlogits is NULL", **{**r, "dlogits": 0})
    refused("route_topk_backward", tg.EINVAL, "overlaps", **{**r, "dlogits": P[0] + 64})
    refused("route_topk_backward", tg.EINVAL, "stride of dlogits", **{**r, "ldo": 8})
    p = dict(T=4096, k=4, E=64, ids=P[0], offsets=P[1], rows=P[2], slots=P[3], workspace=P[4], workspace_bytes=1 << 20)
    refused("route_plan", tg.EINVAL, "E=", **{**p, "E": 1025})
    refused("route_plan", tg.EINVAL, "k=", **{**p, "k": 0})
    refused("route_plan", tg.EINVAL, "workspace bytes", **{**p, "workspace_bytes": 8})
    refused("route_plan", tg.EINVAL, "workspace is NULL", **{**p, "workspace": 0})
    refused("route_plan", tg.EINVAL, "rows overlaps slots", **{**p, "slots": P[2]})
    refused("route_plan", tg.ETOOBIG, "T k", **{**p, "T": 1 << 30})
    g = dict(R=8, D=64, src_rows=4, x=P[0], ldx=64, rows=P[1], out=P[2], ldo=64)
    refused("expert_gather", tg.EALIGN, "multiple of 8", **{**g, "D": 60})
    refused("expert_gather", tg.EINVAL, "out overlaps x", **{**g, "out": P[0]})
    c = dict(dtype=0, T=4, D=64, R=8, k=2, h=P[0], ldh=64, slots=P[1], weights=P[2], out=P[3], ldo=64)
    refused("expert_combine", tg.EINVAL, "element type", **{**c, "dtype": 2})
    refused("expert_combine", tg.EINVAL, "slots is NULL", **{**c, "slots": 0})
    refused("expert_combine", tg.EINVAL, "out overlaps h", **{**c, "out": P[0]})
    refused("expert_combine", tg.EINVAL, "out overlaps residual", **{**c, "residual": P[3] + 16, "ldr": 64})
    b = dict(dtype=0, T=4, D=64, R=8, k=2, dout=P[0], ldd=64, h=P[1], ldh=64, slots=P[2], weights=P[3], dh=P[4],
             ldg=64, dweights=P[5])
    refused("expert_combine_backward", tg.EINVAL, "weights is NULL", **{**b, "weights": 0})
    refused("expert_combine_backward", tg.EINVAL, "dh overlaps h", **{**b, "dh": P[1]})


def test_set_tile_refuses_unknown_tiles():
    for bad in ((32, 32), (256, 128), (192, 192), (-1, -1)):
        with pytest.raises(tg.TgemmError) as e:
            ffn.set_tile(*bad)
        assert e.value.code == tg.EINVAL
    ffn.set_tile()


def test_workspace_sizes():
    L = ffn.lib()
    epilogue = L.tgemm_epilogue_workspace_bytes
    assert epilogue(0, 1, 16, 32, 8192) == 16 * 16 * 32 * 4
    assert epilogue(0, 0, 72, 1024, 2056) == 4 * 72 * 1024 * 4    # 33 slices, 8 or more a split
    assert epilogue(0, 0, 72, 1024, 2048) == 0                    # not deep enough
    assert epilogue(0, 1, 16, 32, 4096) == 0                      # few rows split K by themselves
    assert epilogue(1, 1, 16, 32, 4096) == 8 * 16 * 32 * 4
    assert epilogue(0, 1, 1024, 576, 1 << 20) == 0                # enough tiles without
    assert epilogue(0, 1, 1024, 512, 1 << 20) == 2 * 1024 * 512 * 4
    assert epilogue(0, 1, 0, 32, 8192) == epilogue(0, 1, 16, -8, 8192) == epilogue(0, 1, 16, 1 << 31, 8192) == 0
    assert epilogue(0, 1, 16, 32, 1 << 31) == 0
    assert L.tgemm_epilogue_backward_workspace_bytes(128, 64, 0) == 2 * 64 * 4
    assert L.tgemm_epilogue_backward_workspace_bytes(129, 64, 5) == (3 + 5) * 64 * 4
    assert L.tgemm_epilogue_backward_workspace_bytes(2, 64, 5) == (1 + 2) * 64 * 4
    assert L.tgemm_epilogue_backward_workspace_bytes(-1, 64, 5) == 0
    assert L.tgemm_route_plan_workspace_bytes(8, 8, 64) == 0
    assert L.tgemm_route_plan_workspace_bytes(4097, 1, 64) == 2 * 64 * 4
    assert L.tgemm_route_plan_workspace_bytes(1 << 30, 64, 64) == 0


def test_the_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(8, 8, dtype=torch.bfloat16)
    for f in (lambda: tg.gemm_epilogue(x, x), lambda: tg.epilogue_backward(x, x, "relu"),
              lambda: tg.gemm_grouped(x, x[None], torch.zeros(2, dtype=torch.int32)),
              lambda: tg.gemm_grouped_tn(x, x, torch.zeros(2, dtype=torch.int32)), lambda: tg.route_topk(x, 2),
              lambda: tg.route_plan(torch.zeros(2, 2, dtype=torch.int32), 4),
              lambda: tg.expert_gather(x, torch.zeros(2, dtype=torch.int32)),
              lambda: tg.expert_combine(x, torch.zeros(2, 2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(TypeError):
        tg.gemm_epilogue([[1.0]], x)


def test_the_products_kernels_keep_their_accumulators_in_registers(tmp_path):
    """No kernel of the products uses scratch memory: spilled accumulators cost
    their speed, and the compiler has lost one of them on the way back."""
    tools = "/opt/rocm/lib/llvm/bin"
    if not os.path.exists(os.path.join(tools, "llvm-readelf")):
        pytest.skip("no LLVM tools")
    so = tmp_path / "lib.so"
    so.write_bytes(open(ffn.LIB_PATH, "rb").read())
    subprocess.run([os.path.join(tools, "llvm-objdump"), "--offloading", str(so)], capture_output=True, check=True,
                   cwd=tmp_path)
    seen = 0
    for f in tmp_path.glob("lib.so.*gfx950*"):
        notes = subprocess.run([os.path.join(tools, "llvm-readelf"), "--notes", str(f)], capture_output=True, text=True,
                               check=True).stdout
        for name, size in re.findall(r"\.name:\s+(\S+).*?\.private_segment_fixed_size:\s+(\d+)", notes, re.S):
            if re.search(r"(epilogue|grouped|grouped_tn|rows)_kernel", name):
                seen += 1
                assert int(size) == 0, name
    assert seen > 60


def test_the_k_splits_kernels_keep_their_accumulators_in_registers(tmp_path):
    """The same of the K split: its products and the kernel that joins their
    sums, which are no instances of the epilogue's."""
    tools = "/opt/rocm/lib/llvm/bin"
    if not os.path.exists(os.path.join(tools, "llvm-readelf")):
        pytest.skip("no LLVM tools")
    so = tmp_path / "lib.so"
    so.write_bytes(open(ffn.LIB_PATH, "rb").read())
    subprocess.run([os.path.join(tools, "llvm-objdump"), "--offloading", str(so)], capture_output=True, check=True,
                   cwd=tmp_path)
    seen = {"split": 0, "join": 0}
    for f in tmp_path.glob("lib.so.*gfx950*"):
        notes = subprocess.run([os.path.join(tools, "llvm-readelf"), "--notes", str(f)], capture_output=True, text=True,
                               check=True).stdout
        for name, size in re.findall(r"\.name:\s+(\S+).*?\.private_segment_fixed_size:\s+(\d+)", notes, re.S):
            kind = re.search(r"\d(split|join)_kernel", name)
            if kind:
                seen[kind.group(1)] += 1
                assert int(size) == 0, name
    assert seen == {"split": 8, "join": 4}        # types and layouts; types, gated or not
