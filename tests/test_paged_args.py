"""Refusals of the paged serving calls: everything a call can know from its
arguments is refused on the host before a launch.  No GPU is needed."""
import ctypes

import pytest

import kv_cache_compression_cachegen_b200 as cg

SHAPE = cg.Shape(4, 2, 64)


@pytest.fixture(autouse=True)
def _built(native_built):
    return native_built


def _extend(**kw):
    a = cg.ExtendArgs()
    vals = dict(num_requests=4, page_tokens=16, num_pages=64, max_pages=8, num_free=10,
                max_tokens=32, position_base=0, held=256, added=256, free_pages=256, taken=256,
                taken_out=256, block_tables=256, kv_lens=256, q_starts=256, slots=256,
                positions=256, status=256)
    vals.update(kw)
    for k, v in vals.items():
        setattr(a, k, v)
    return cg.cg_extend_tables(a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(num_requests=0), dict(page_tokens=0), dict(num_pages=0), dict(max_pages=0),
    dict(num_free=-1), dict(max_tokens=0), dict(position_base=-1), dict(held=None),
    dict(added=None), dict(free_pages=None), dict(taken=None), dict(taken_out=None),
    dict(block_tables=None), dict(kv_lens=None), dict(q_starts=None), dict(slots=None),
    dict(slots=260), dict(positions=None), dict(status=None), dict(held=258)])
def test_extend_tables_refusals(bad):
    assert _extend(**bad) == cg.CG_ERR_INVALID_ARG


def test_extend_tables_limit():
    assert _extend(num_requests=8193) == cg.CG_ERR_UNSUPPORTED


def _append(shape=SHAPE, **kw):
    a = cg.AppendArgs()
    vals = dict(num_tokens=5, num_q_heads=4, layer=1, num_pages=64, page_tokens=16,
                max_positions=100, rot_dim=64, interleaved=0, dtype=0, eps=1e-6, q=256, k=256,
                v=256, q_stride=512, k_stride=512, v_stride=512, q_out=4096, q_out_stride=256,
                q_weight=None, k_weight=None, rope=256, positions=256, slots=256, pool=256,
                status=256)
    vals.update(kw)
    for k, v in vals.items():
        setattr(a, k, v)
    return cg.cg_append_qkv(shape, a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(num_tokens=0), dict(num_q_heads=3), dict(num_q_heads=0), dict(layer=4), dict(layer=-1),
    dict(num_pages=0), dict(page_tokens=0), dict(max_positions=0), dict(rot_dim=63),
    dict(rot_dim=66), dict(rot_dim=-2), dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")),
    dict(q=None), dict(q=264), dict(k=None), dict(v=None), dict(q_out=None), dict(q_stride=255),
    dict(q_stride=260), dict(k_stride=120), dict(v_stride=0), dict(q_out_stride=248),
    dict(q_weight=8), dict(k_weight=8), dict(rope=None), dict(positions=None), dict(slots=None),
    dict(slots=4), dict(pool=None), dict(pool=8), dict(status=None), dict(q_out=256)])
def test_append_refusals(bad):
    assert _append(**bad) == cg.CG_ERR_INVALID_ARG


def test_append_limits():
    assert _append(shape=cg.Shape(4, 2, 40)) == cg.CG_ERR_UNSUPPORTED
    assert _append(num_q_heads=130) == cg.CG_ERR_UNSUPPORTED
    assert _append(num_pages=1 << 28, page_tokens=16) == cg.CG_ERR_UNSUPPORTED
    assert _append(num_tokens=1 << 30) == cg.CG_ERR_UNSUPPORTED


def _attention(shape=SHAPE, prefix=None, **kw):
    a = cg.AttentionArgs()
    vals = dict(num_requests=2, num_tokens=5, max_q=3, num_q_heads=4, layer=1, num_pages=64,
                page_tokens=16, max_pages=8, window=0, sinks=0, dtype=0, scale=0.125, q=256,
                out=4096, q_stride=256, out_stride=256, lse=None, q_starts=256, kv_lens=256,
                block_tables=256, pool=256, status=256, workspace=256,
                workspace_bytes=cg.cg_attention_workspace_bytes(SHAPE, 4, 5, 2, True))
    vals.update(kw)
    for k, v in vals.items():
        setattr(a, k, v)
    if prefix is None:
        return cg.cg_attention_paged(shape, a, stream=0)
    return cg.cg_attention_shared(shape, a, *prefix, stream=0)


BAD_ATTENTION = [
    dict(num_requests=0), dict(num_tokens=0), dict(max_q=0), dict(num_q_heads=3), dict(layer=4),
    dict(num_pages=0), dict(page_tokens=0), dict(max_pages=0), dict(dtype=-1),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(q=None), dict(q=264), dict(out=None),
    dict(out=256), dict(q_stride=248), dict(out_stride=257), dict(lse=2), dict(q_starts=None),
    dict(kv_lens=None), dict(block_tables=None), dict(pool=None), dict(status=None),
    dict(workspace=None), dict(workspace=128), dict(window=-1), dict(sinks=-1)]


@pytest.mark.parametrize("bad", BAD_ATTENTION)
def test_attention_refusals(bad):
    assert _attention(**bad) == cg.CG_ERR_INVALID_ARG
    assert _attention(prefix=(256, 100), **bad) == cg.CG_ERR_INVALID_ARG


def test_attention_limits_and_workspace():
    need = cg.cg_attention_workspace_bytes(SHAPE, 4, 5, 2)
    assert need <= cg.cg_attention_workspace_bytes(SHAPE, 4, 5, 2, True)
    assert _attention(workspace_bytes=need - 1) == cg.CG_ERR_CAPACITY
    assert _attention(num_requests=8193) == cg.CG_ERR_UNSUPPORTED
    assert _attention(num_pages=1 << 28) == cg.CG_ERR_UNSUPPORTED
    assert _attention(shape=cg.Shape(4, 2, 272)) == cg.CG_ERR_UNSUPPORTED
    assert _attention(prefix=(None, 100)) == cg.CG_ERR_INVALID_ARG
    assert _attention(prefix=(256, -1)) == cg.CG_ERR_INVALID_ARG
    assert _attention(prefix=(256, 2 ** 31 - 1)) == cg.CG_ERR_UNSUPPORTED
    # the shared form has no window
    assert _attention(prefix=(256, 100), window=8) == cg.CG_ERR_INVALID_ARG
    assert _attention(prefix=(256, 100), sinks=1) == cg.CG_ERR_INVALID_ARG
    lib = cg.library()
    assert lib.cg_attention_paged(ctypes.byref(SHAPE), None, None) == cg.CG_ERR_INVALID_ARG
    assert lib.cg_append_qkv(ctypes.byref(SHAPE), None, None) == cg.CG_ERR_INVALID_ARG
    assert lib.cg_extend_tables(None, None) == cg.CG_ERR_INVALID_ARG
    out = ctypes.c_uint64()
    assert lib.cg_attention_workspace_bytes(ctypes.byref(SHAPE), 4, 0, 2, 0,
                                            ctypes.byref(out)) == cg.CG_ERR_INVALID_ARG


def test_rope_table_refusals():
    for args in ((0, 64, 1e4, 256), (8, 63, 1e4, 256), (8, 0, 1e4, 256), (8, 64, 0.0, 256),
                 (8, 64, float("inf"), 256), (8, 64, 1e4, None)):
        assert cg.cg_rope_table(*args, stream=0) == cg.CG_ERR_INVALID_ARG
    assert cg.cg_rope_table(8, 258, 1e4, 256, stream=0) == cg.CG_ERR_UNSUPPORTED


def test_argument_blocks_match_the_header():
    # field by field, in order: the ctypes blocks mirror the C structs
    import re
    from pathlib import Path
    text = (Path(__file__).resolve().parents[1] / "include" / "cachegen.h").read_text("utf-8")
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, block in (("cg_extend_args", cg.ExtendArgs), ("cg_append_args", cg.AppendArgs),
                        ("cg_attention_args", cg.AttentionArgs)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        fields = []
        for decl in body.split(";"):
            decl = decl.strip()
            if not decl:
                continue
            names = re.sub(r"^(const\s+)?\w+\s*\*?\s*", "", decl)
            pointer = "*" in decl
            for n in names.split(","):
                n = n.strip().lstrip("*").strip()
                fields.append((n[:-4] if n.endswith("_dev") else n, pointer or n.endswith("_dev"),
                               decl.split()[0]))
        mirror = [(n, t is ctypes.c_void_p) for n, t in block._fields_]
        assert [(n, p) for n, p, _ in fields] == mirror, name
        wide = {"int64_t", "uint64_t"}
        for (n, p, c), (_, t) in zip(fields, block._fields_):
            assert ctypes.sizeof(t) == (8 if p or c in wide else 4), (name, n)
