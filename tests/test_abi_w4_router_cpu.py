"""Refusals and size helpers of the 4-bit layer and of the router's training
entry points, and the packed 4-bit layout, on a machine without a GPU.

No call here enqueues device work: each is pure host code or must be rejected
by validation before any HIP call."""
import ctypes
import os
import re
import subprocess

import pytest

from mixture_experts_layer_up_amd import binding, build
from mixture_experts_layer_up_amd.synth import CONFIGS

INVALID, SHAPE, WS, ALIGN = -1, -2, -3, -4
ref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        build.build(verbose=False)
    return binding.load_library()


def _p(addr=4096):
    return ctypes.c_void_p(addr)   # never dereferenced: validation rejects first


def _shape(**over):
    return binding.make_shape(CONFIGS["decode64"].replace(**over))


@pytest.mark.parametrize("cname,cls", [
    ("moe_lora_w4_format", "W4Format"), ("moe_lora_w4_weights", "W4Weights"),
    ("moe_lora_tokens", "Tokens"), ("moe_lora_balance", "Balance")])
def test_ctypes_structs_match_header(cname, cls):
    text = re.sub(r"/\*.*?\*/", "", open(binding.HEADER_PATH).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (cname, cname), text, re.S).group(1)
    fields = [(re.search(r"(\w+)\s*$", d).group(1), "*" in d) for d in body.split(";") if d.strip()]
    assert fields == [(n, t is ctypes.c_void_p) for n, t in getattr(binding, cls)._fields_]


@pytest.mark.parametrize("group,zeros,rc", [(0, 0, SHAPE), (16, 0, SHAPE), (48, 0, SHAPE), (256, 1, SHAPE),
                                            (-32, 0, SHAPE), (64, 2, INVALID), (64, -1, INVALID)])
def test_bad_formats(lib, group, zeros, rc):
    shape, fmt = _shape(), binding.W4Format(group, zeros)
    assert binding.workspace_size_w4(shape, fmt) == 0
    assert binding.packed_w4_bytes(shape, fmt, 0) == 0
    q = binding.W4Weights(4096, 4096, 4096 if zeros else None)
    inp = binding.Inputs()
    assert lib.moe_lora_pack_weights_w4(ref(shape), ref(fmt), ref(q), ref(q), _p(), _p(), None) == rc
    assert lib.moe_lora_quantize_w4(ref(shape), ref(fmt), _p(), _p(), ref(q), ref(q), None) == rc
    assert lib.moe_lora_forward_w4(ref(shape), ref(fmt), ref(inp), None, _p(), _p(), 1 << 40, None) == rc


def test_null_format_and_bad_shape(lib):
    shape, fmt = _shape(), binding.W4Format(64, 0)
    inp = binding.Inputs()
    assert lib.moe_lora_workspace_size_w4(ref(shape), None) == 0
    assert lib.moe_lora_packed_w4_bytes(ref(shape), ref(fmt), 2) == 0
    assert lib.moe_lora_forward_w4(ref(shape), None, ref(inp), None, _p(), _p(), 1 << 40, None) == INVALID
    assert lib.moe_lora_forward_w4(ref(shape), ref(fmt), None, None, _p(), _p(), 1 << 40, None) == INVALID
    bad = _shape(hidden=96)
    assert binding.workspace_size_w4(bad, fmt) == 0
    assert lib.moe_lora_forward_w4(ref(bad), ref(fmt), ref(inp), None, _p(), _p(), 1 << 40, None) == SHAPE


@pytest.mark.parametrize("H,I,group,zeros", [(2048, 768, 128, 0), (64, 32, 32, 1), (1088, 416, 64, 1)])
def test_packed_bytes(lib, H, I, group, zeros):
    """Codes in whole steps of 128 rows, a bf16 scale and a zero-point byte per group and column."""
    shape = _shape(hidden=H, inter=I)
    fmt = binding.W4Format(group, zeros)
    for which, (K, N) in enumerate(((H, 2 * I), (I, H))):
        want = 128 * N * (-(-K // 128) * 64 + -(-K // group) * (2 + zeros))
        assert binding.packed_w4_bytes(shape, fmt, which) == want


def test_w4_pack_and_quantize_arguments(lib):
    shape, fmt = _shape(), binding.W4Format(64, 1)
    W = binding.W4Weights
    ok = W(4096, 4096, 4096)
    pack = lambda a, b, c=_p(), d=_p(): lib.moe_lora_pack_weights_w4(  # noqa: E731
        ref(shape), ref(fmt), a, b, c, d, None)
    assert pack(None, ref(ok)) == INVALID and pack(ref(ok), None) == INVALID
    assert pack(ref(ok), ref(ok), None) == INVALID and pack(ref(ok), ref(ok), _p(), None) == INVALID
    for q, rc in ((W(None, 4096, 4096), INVALID), (W(4096, None, 4096), INVALID),
                  (W(4096, 4096, None), INVALID), (W(4096, 4097, 4096), ALIGN)):
        assert pack(ref(q), ref(ok)) == rc and pack(ref(ok), ref(q)) == rc
        assert lib.moe_lora_quantize_w4(ref(shape), ref(fmt), _p(), _p(), ref(q), ref(ok), None) == rc
    plain = binding.W4Format(64, 0)     # zero points given to a format without them
    assert lib.moe_lora_pack_weights_w4(ref(shape), ref(plain), ref(ok), ref(ok), _p(), _p(), None) == INVALID
    assert pack(ref(ok), ref(ok), _p(4096 + 8)) == ALIGN and pack(ref(ok), ref(ok), _p(), _p(4104)) == ALIGN
    quant = lambda a, b: lib.moe_lora_quantize_w4(ref(shape), ref(fmt), a, b, ref(ok), ref(ok), None)  # noqa: E731
    assert quant(None, _p()) == INVALID and quant(_p(), None) == INVALID and quant(_p(4097), _p()) == ALIGN


def _inputs(**over):
    base = {n: 4096 for n in ("hidden", "router_logits", "w13_packed", "w2_packed", "lora_a_gate_up",
                              "lora_b_gate_up", "lora_a_down", "lora_b_down", "token_lora_mapping")}
    base.update(over)
    return binding.Inputs(*[base.get(n) for n, _ in binding.Inputs._fields_])


@pytest.mark.parametrize("over,rc", [
    (dict(hidden=None), INVALID), (dict(w13_packed=None), INVALID), (dict(w2_packed=4104), ALIGN),
    (dict(topk_ids=4096, topk_weights=4096), INVALID), (dict(router_logits=None, topk_ids=4096), INVALID),
    (dict(lora_b_gate_up=None), INVALID), (dict(expert_out=4096), INVALID), (dict(side_stream=4096), INVALID)])
def test_forward_w4_arguments(lib, over, rc):
    shape, fmt = _shape(), binding.W4Format(128, 0)
    need = binding.workspace_size_w4(shape, fmt)
    call = lambda inp, ws, n, out=_p(): lib.moe_lora_forward_w4(  # noqa: E731
        ref(shape), ref(fmt), ref(inp), None, out, ws, n, None)
    assert call(_inputs(**over), _p(1 << 20), need) == rc
    assert call(_inputs(), _p(1 << 20), need - 1) == WS
    assert call(_inputs(), _p((1 << 20) + 16), need) == ALIGN
    assert call(_inputs(), None, need) == INVALID
    assert call(_inputs(), _p(1 << 20), need, None) == INVALID


def test_workspace_w4_is_monotone(lib):
    fmt = binding.W4Format(128, 0)
    sizes = [binding.workspace_size_w4(_shape(num_tokens=T), fmt) for T in (0, 1, 64, 512, 4096)]
    assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)
    # fp32 expert outputs and bf16 activations of every slot
    assert sizes[-1] >= 4096 * 8 * (2048 * 4 + 768 * 2)


def _balance(**over):
    base = dict(loss=4096, expert_counts=4096, expert_probs=4096, seq_tokens=4096)
    base.update(over)
    return binding.Balance(*[base[n] for n, _ in binding.Balance._fields_])


def test_balance_loss_arguments(lib):
    shape = _shape(num_tokens=2048)
    need = lib.moe_lora_balance_workspace_size(ref(shape), 4)
    assert need > 0 and lib.moe_lora_balance_workspace_size(ref(shape), 8) >= need
    assert lib.moe_lora_balance_workspace_size(ref(_shape()), 1) == 0       # a small batch
    for bad in (0, -1, 65536):
        assert lib.moe_lora_balance_workspace_size(ref(shape), bad) == 0
    assert lib.moe_lora_balance_workspace_size(ref(_shape(top_k=0)), 1) == 0

    def call(logits=_p(), ids=_p(), tokens=None, bal=_balance(), ws=_p(1 << 20), n=1 << 40, s=shape):
        t = ref(tokens) if tokens is not None else None
        return lib.moe_lora_balance_loss(ref(s), logits, ids, t, ref(bal) if bal is not None else None,
                                         ws, n, None)

    assert call(logits=None) == INVALID and call(ids=None) == INVALID and call(bal=None) == INVALID
    for name in ("loss", "expert_counts", "expert_probs", "seq_tokens"):
        assert call(bal=_balance(**{name: None})) == INVALID
    assert call(ws=None) == INVALID and call(n=16) == WS and call(ws=_p((1 << 20) + 64)) == ALIGN
    T = binding.Tokens
    assert call(tokens=T(None, 4096, 0)) == SHAPE and call(tokens=T(None, 4096, 65536)) == SHAPE
    assert call(tokens=T(4096, None, 2)) == INVALID
    assert call(tokens=T(None, 4096, 4), n=need - 1) == WS
    assert call(s=_shape(num_experts=2048)) == SHAPE
    assert lib.moe_lora_balance_loss(None, _p(), _p(), None, ref(_balance()), None, 0, None) == INVALID


def test_route_backward_arguments(lib):
    def call(logits=_p(), ids=_p(), w=_p(), dw=_p(), tokens=None, bal=_balance(), d_loss=_p(), out=_p(),
             s=_shape()):
        return lib.moe_lora_route_backward(ref(s), logits, ids, w, dw,
                                           ref(tokens) if tokens is not None else None,
                                           ref(bal) if bal is not None else None, d_loss, out, None)

    assert call(out=None) == INVALID and call(d_loss=None) == INVALID and call(bal=None) == INVALID
    assert call(dw=None, bal=None, d_loss=None) == INVALID                     # neither part
    assert call(ids=None) == INVALID and call(w=None) == INVALID
    assert call(logits=None) == INVALID
    assert call(logits=None, bal=None, d_loss=None, s=_shape(routing_method=1)) == INVALID
    assert call(bal=_balance(expert_counts=None)) == INVALID
    assert call(bal=_balance(seq_tokens=None)) == INVALID
    assert call(tokens=binding.Tokens(None, None, 3)) == INVALID
    assert call(tokens=binding.Tokens(None, 4096, 0)) == SHAPE
    assert call(s=_shape(top_k=0)) == SHAPE
    # an empty batch has no gradient rows
    assert call(logits=None, ids=None, w=None, dw=None, bal=None, d_loss=None, out=None,
                s=_shape(num_tokens=0)) == 0


def test_finalize_backward_arguments(lib):
    def call(d=_p(), y=_p(), perm=_p(), w=_p(), dy=_p(), dw=_p(), s=_shape()):
        return lib.moe_lora_finalize_backward(ref(s), d, y, perm, w, dy, dw, None)

    assert call(d=None) == INVALID and call(perm=None) == INVALID and call(dy=None, dw=None) == INVALID
    assert call(y=None) == INVALID and call(w=None) == INVALID
    assert call(d=_p(4104)) == ALIGN and call(y=_p(4104)) == ALIGN and call(dy=_p(4098)) == ALIGN
    assert call(s=_shape(inter=48)) == SHAPE
    assert call(None, None, None, None, None, None, _shape(num_tokens=0)) == 0


LAYOUT = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "w4_layout.h"
using namespace moe_lora;

// args: E K N I group zeros.  Every weight has one nibble of its own inside the
// codes region, every (group, column) one scale and one zero point.
int main(int, char **v)
{
    const int E = atoi(v[1]), K = atoi(v[2]), N = atoi(v[3]), I = atoi(v[4]), group = atoi(v[5]);
    const W4Layout l = w4_layout(E, K, N, group, atoi(v[6]) != 0);
    std::vector<unsigned char> bit(l.scales * 8), col(N);
    for (int slab = 0; slab < l.n_slabs; ++slab)
        for (int t = 0; t < 4; ++t)
            for (int c = 0; c < 16; ++c) {
                const int n = w4_column(slab, t, c, I);
                if (n < 0 || n >= N || col[n]++) return puts("column twice"), 1;
            }
    for (int n = 0; n < N; ++n)
        if (col[n] != 1) return puts("column missing"), 1;
    for (int e = 0; e < E; ++e)
        for (int slab = 0; slab < l.n_slabs; ++slab)
            for (int t = 0; t < 4; ++t)
                for (int c = 0; c < 16; ++c)
                    for (int k = 0; k < K; ++k) {
                        const int u = k / 64, chunk = (k / 32) & 1, lane = ((k / 8) & 3) * 16 + c;
                        const size_t word = (((size_t)e * l.n_slabs + slab) * l.k_units + u) * 512 +
                                            (size_t)(t / 2) * 256 + lane * 4 + (t & 1) * 2 + chunk;
                        for (int b = 0; b < 4; ++b) {
                            const size_t at = word * 32 + ((w4_nibble_bit(k & 7) + b) & 31);
                            if (at >= bit.size() || bit[at]++) return puts("bit twice or outside"), 1;
                        }
                    }
    // after rotating right by 4 j, rows 2j and 2j + 1 sit at bits 3 and 19
    for (int i = 0; i < 8; ++i)
        if (((w4_nibble_bit(i) - 4 * (i / 2)) & 31) != (i & 1 ? 19 : 3)) return puts("nibble"), 1;
    if (l.scales % 16 || (l.zeros - l.scales) != (size_t)E * l.n_slabs * l.n_groups * 128) return 1;
    puts("ok");
    return 0;
}
"""


@pytest.fixture(scope="module")
def layout_program(tmp_path_factory):
    d = tmp_path_factory.mktemp("w4_layout")
    (d / "layout.cpp").write_text(LAYOUT)
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{build.CSRC}", str(d / "layout.cpp"), "-o",
                    str(d / "layout")], check=True, capture_output=True)
    return str(d / "layout")


@pytest.mark.parametrize("E,K,N,I,group,zeros", [
    (2, 128, 128, 64, 32, 1), (3, 96, 192, 0, 64, 0), (1, 32, 64, 32, 128, 1), (1, 416, 320, 0, 128, 1)])
def test_packed_layout_is_one_to_one(layout_program, E, K, N, I, group, zeros):
    r = subprocess.run([layout_program, *map(str, (E, K, N, I, group, zeros))], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
