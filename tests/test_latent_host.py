"""CPU tests of the latent-attention and step-metadata calls: what their C entry points and the
Python binding refuse on the host, before any device work."""
import ctypes

import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from pagedattention_paged_kv_gb300 import _build

INVALID, UNSUPPORTED = -1, -2
SOME = ctypes.c_void_p(4096)   # an aligned address that nothing dereferences
NULL = ctypes.c_void_p(0)
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return pkv.lib()


def call(f, defaults, **changes):
    """f over the defaults (an ordered dict of its arguments) with some of them changed."""
    assert set(changes) <= set(defaults)
    return f(*{**defaults, **changes}.values())


STEP = dict(block_tables=SOME, context_lens=SOME, query_start_loc=SOME, slot_mapping=SOME, free_end=SOME,
            cached_lens=SOME, new_lens=SOME, free_blocks=SOME, free_begin=SOME, num_seqs=4, max_blocks=8,
            num_slots=64, num_free=16, num_blocks=32, block_size=16, stream=NULL)


@pytest.mark.parametrize("changes,status", [
    (dict(num_seqs=-1), INVALID), (dict(max_blocks=-1), INVALID), (dict(num_slots=-1), INVALID),
    (dict(num_free=-1), INVALID), (dict(num_blocks=-1), INVALID), (dict(block_size=0), INVALID),
    (dict(block_size=12), UNSUPPORTED), (dict(block_size=128), UNSUPPORTED),
    (dict(num_seqs=16385), UNSUPPORTED), (dict(num_slots=2 ** 31), UNSUPPORTED),
    (dict(num_free=2 ** 31), UNSUPPORTED), (dict(num_blocks=2 ** 31), UNSUPPORTED),
    (dict(max_blocks=2 ** 27), UNSUPPORTED),
    (dict(block_tables=NULL), INVALID), (dict(context_lens=NULL), INVALID),
    (dict(query_start_loc=NULL), INVALID), (dict(slot_mapping=NULL), INVALID), (dict(free_end=NULL), INVALID),
    (dict(cached_lens=NULL), INVALID), (dict(new_lens=NULL), INVALID), (dict(free_blocks=NULL), INVALID),
    (dict(free_begin=NULL), INVALID), (dict(slot_mapping=ctypes.c_void_p(4100)), INVALID)])
def test_step_metadata_refuses(lib, changes, status):
    assert call(lib.pkv_step_metadata, STEP, **changes) == status


WRITE = dict(cache=SOME, latent=SOME, rope=SOME, slots=SOME, num_tokens=3, num_blocks=4, block_size=16,
             latent_dim=512, rope_dim=64, dtype=0, stream=NULL)
ODD = ctypes.c_void_p(4104)


@pytest.mark.parametrize("changes,status", [
    (dict(num_tokens=-1), INVALID), (dict(num_blocks=-1), INVALID), (dict(block_size=0), INVALID),
    (dict(latent_dim=0), INVALID), (dict(rope_dim=-8), INVALID),
    (dict(dtype=1), UNSUPPORTED), (dict(latent_dim=508), UNSUPPORTED), (dict(rope_dim=60), UNSUPPORTED),
    (dict(latent_dim=65544), UNSUPPORTED), (dict(num_blocks=2 ** 31), UNSUPPORTED),
    (dict(cache=NULL), INVALID), (dict(latent=NULL), INVALID), (dict(rope=NULL), INVALID),
    (dict(slots=NULL), INVALID), (dict(cache=ODD), INVALID), (dict(latent=ODD), INVALID),
    (dict(rope=ODD), INVALID), (dict(slots=ctypes.c_void_p(4100)), INVALID),
    (dict(num_tokens=0, cache=NULL, latent=NULL, rope=NULL, slots=NULL), 0)])
def test_latent_cache_write_refuses(lib, changes, status):
    assert call(lib.pkv_latent_cache_write, WRITE, **changes) == status


ABSORBED = dict(out=SOME, q=SOME, query_start_loc=NULL, cache=SOME, tables=SOME, ctx=SOME, num_seqs=3, total_q=3,
                max_blocks=4, num_heads=16, latent_dim=512, rope_dim=64, block_size=16, num_blocks=32, scale=F(0.1),
                causal=1, dtype=0, workspace=SOME, workspace_bytes=ctypes.c_size_t(0), stream=NULL)
# what both forms refuse alike
COMMON = [
    (dict(num_seqs=-1), INVALID), (dict(total_q=-1), INVALID), (dict(max_blocks=-1), INVALID),
    (dict(num_heads=0), INVALID), (dict(latent_dim=0), INVALID), (dict(rope_dim=0), INVALID),
    (dict(block_size=0), INVALID), (dict(num_blocks=-1), INVALID),
    (dict(dtype=1), UNSUPPORTED), (dict(latent_dim=384), UNSUPPORTED), (dict(rope_dim=32), UNSUPPORTED),
    (dict(block_size=12), UNSUPPORTED), (dict(block_size=128), UNSUPPORTED),
    (dict(num_blocks=2 ** 31), UNSUPPORTED), (dict(max_blocks=2 ** 27), UNSUPPORTED),
    (dict(scale=F(0.0)), INVALID), (dict(scale=F(-1.0)), INVALID), (dict(scale=F(float("nan"))), INVALID),
    (dict(scale=F(float("inf"))), INVALID),
    (dict(out=NULL), INVALID), (dict(q=NULL), INVALID), (dict(cache=NULL), INVALID), (dict(tables=NULL), INVALID),
    (dict(ctx=NULL), INVALID), (dict(out=ODD), INVALID), (dict(q=ODD), INVALID), (dict(cache=ODD), INVALID),
    (dict(num_blocks=0), INVALID), (dict(max_blocks=0), INVALID),
    (dict(num_seqs=0, total_q=0, out=NULL, q=NULL, cache=NULL, tables=NULL, ctx=NULL), 0)]


@pytest.mark.parametrize("changes,status", COMMON + [
    (dict(total_q=4), INVALID),    # one row a sequence without offsets
    (dict(total_q=2 ** 27, num_heads=16, query_start_loc=SOME), UNSUPPORTED)])
def test_latent_attention_absorbed_refuses(lib, changes, status):
    assert call(lib.pkv_latent_attention_absorbed, ABSORBED, **changes) == status


EXPANDED = dict(out=SOME, q=SOME, query_start_loc=SOME, cache=SOME, tables=SOME, ctx=SOME, w_k=SOME, w_v=SOME,
                num_seqs=3, total_q=300, total_context=1000, max_blocks=64, num_heads=16, latent_dim=512, rope_dim=64,
                nope_dim=128, v_dim=128, block_size=16, num_blocks=256, scale=F(0.1), causal=1, dtype=0,
                workspace=SOME, workspace_bytes=ctypes.c_size_t(0), stream=NULL)


@pytest.mark.parametrize("changes,status", COMMON + [
    (dict(query_start_loc=NULL), INVALID), (dict(w_k=NULL), INVALID), (dict(w_v=NULL), INVALID),
    (dict(w_k=ODD), INVALID), (dict(w_v=ODD), INVALID), (dict(out=ctypes.c_void_p(4112)), INVALID),
    (dict(total_context=-1), INVALID), (dict(nope_dim=0), INVALID), (dict(v_dim=-1), INVALID),
    (dict(nope_dim=64), UNSUPPORTED), (dict(v_dim=256), UNSUPPORTED),
    (dict(total_context=2 ** 25), UNSUPPORTED),          # 16 heads x 2^25 rows
    (dict(total_context=2 ** 63 - 1), UNSUPPORTED),      # a sum past 63 bits
    (dict(total_q=1, num_heads=2 ** 31 - 200, total_context=2 ** 31 - 1, num_seqs=2 ** 31 - 1), UNSUPPORTED)])
def test_latent_attention_expanded_refuses(lib, changes, status):
    assert call(lib.pkv_latent_attention_expanded, EXPANDED, **changes) == status


@pytest.mark.parametrize("args", [
    (7, 1, 1, 0, 16, 512, 64), (3, 1, 1, -1, 16, 512, 64), (3, 1, 1, 2 ** 63 - 1, 16, 512, 64),
    (3, 2 ** 31 - 1, 0, 2 ** 31 - 1, 2 ** 31 - 1, 512, 64), (2, -1, 1, 0, 16, 512, 64), (2, 1, 1, 0, 0, 512, 64),
    (2, 1, 1, 0, 16, 128, 64), (2, 1, 1, 0, 16, 512, 128)])
def test_latent_workspace_size_is_zero_for_what_is_unsupported(lib, args):
    assert lib.pkv_latent_workspace_size(*args) == 0


def test_the_binding_refuses_host_tensors():
    b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="block_tables"):
        pkv.step_metadata(i32(2, 4), i32(2), i32(3), torch.zeros(8, dtype=torch.int64), i32(1), i32(2), i32(2),
                          i32(8), i32(1), 8)
    with pytest.raises(ValueError, match="latent_cache"):
        pkv.latent_cache_write(b16(2, 16, 576), b16(3, 512), b16(3, 64), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="q must be"):
        pkv.latent_attention_absorbed(b16(2, 4, 512), b16(2, 4, 576), b16(2, 16, 576), i32(2, 1), i32(2), 0.1)
    with pytest.raises(ValueError, match="q must be"):
        pkv.latent_attention_expanded(b16(2, 4, 128), b16(2, 4, 192), i32(2), b16(2, 16, 576), i32(1, 1), i32(1),
                                      b16(4, 128, 512), b16(4, 128, 512), 0.1, 2)
    with pytest.raises(ValueError, match="query_start_loc"):
        pkv.latent_attention_expanded(b16(2, 4, 128), b16(2, 4, 192), None, b16(2, 16, 576), i32(1, 1), i32(1),
                                      b16(4, 128, 512), b16(4, 128, 512), 0.1, 2)
