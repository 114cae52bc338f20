"""The packed, shared-prefix, append and eviction calls from a strict C99 program: parameter
layouts, workspace sizes and host-side refusals (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

from block_sparse_attention_lva_b200 import _binding as lb
from tests.test_c_header import CUDA_INCLUDE, INCLUDE, PKG

PROGRAM = r"""
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#include "lva.h"

int main(void) {
  lva_packed_params p;
  lva_shared_prefix_params x;
  void* a = (void*)(uintptr_t)256;
  int32_t* i = (int32_t*)(uintptr_t)256;
  int32_t* i2 = (int32_t*)(uintptr_t)260;
  float* f = (float*)(uintptr_t)256;
  lva_status s;
  memset(&p, 0, sizeof(p));
  memset(&x, 0, sizeof(x));
  printf("packed %d %d %d\n", (int)sizeof(p), (int)offsetof(lva_packed_params, total_q), (int)offsetof(lva_packed_params, o_head_stride));
  printf("prefix %d %d %d\n", (int)sizeof(x), (int)offsetof(lva_shared_prefix_params, prefix_len),
         (int)offsetof(lva_shared_prefix_params, o_head_stride));
  p.num_seqs = 1; p.q_heads = 40; p.kv_heads = 8; p.d = 128; p.causal = 1; p.scale = 0.09f;
  p.total_q = 64; p.total_k = 8000;
  printf("packed bytes %lld\n", (long long)lva_packed_workspace_bytes(&p));
  s = lva_packed_attn(&p, a, a, a, a, f, i, i, NULL, 0, (cudaStream_t)0);
  printf("strides %s: %s\n", lva_status_string(s), lva_last_error_message());
  p.q_token_stride = p.o_token_stride = 40 * 128; p.k_token_stride = p.v_token_stride = 8 * 128;
  p.q_head_stride = p.k_head_stride = p.v_head_stride = p.o_head_stride = 128;
  s = lva_packed_attn(&p, a, a, a, a, f, i, i, a, 100, (cudaStream_t)0);
  printf("small %s\n", lva_status_string(s));
  p.total_q = 0;
  s = lva_packed_attn(&p, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0, (cudaStream_t)0);
  printf("empty %s\n", lva_status_string(s));
  x.B = 4; x.steps = 1; x.q_heads = 8; x.kv_heads = 2; x.d = 64; x.scale = 0.125f; x.prefix_len = 300; x.capacity = 100;
  printf("prefix bytes %d\n", lva_shared_prefix_workspace_bytes(&x, 1) > lva_shared_prefix_workspace_bytes(&x, 0));
  x.steps = 17;
  printf("rows %lld\n", (long long)lva_shared_prefix_workspace_bytes(&x, 0));
  s = lva_append_cache(a, a, 128, 64, 128, 64, a, a, NULL, i, i2, 2, 1, 2, 50, 64, (cudaStream_t)0);
  printf("append %s: %s\n", lva_status_string(s), lva_last_error_message());
  s = lva_evict_cache(a, a, f, i, a, a, f, i, i, 2, 2, 50, 64, 60, 0, 0, (cudaStream_t)0);
  printf("evict %s: %s\n", lva_status_string(s), lva_last_error_message());
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None or not os.path.isdir(CUDA_INCLUDE), reason="needs gcc and the CUDA headers")
def test_c_program(tmp_path):
    src, exe = tmp_path / "context.c", tmp_path / "context"
    src.write_text(PROGRAM)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", INCLUDE, "-isystem", CUDA_INCLUDE, str(src),
                    "-o", str(exe), "-L", PKG, "-llva", f"-Wl,-rpath,{PKG}"], check=True, capture_output=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    size = lb._PACKED.size
    assert out[0] == f"packed {size} 24 {size - 8}" and out[1] == f"prefix {lb._PREFIX.size} 24 {lb._PREFIX.size - 8}"
    assert int(out[2].split()[-1]) == lb.lva_packed_workspace_bytes(1, 40, 8, 128, 64, 8000) > 0
    assert out[3].startswith("strides LVA_ERR_INVALID_ARG: packed: strides")
    assert out[4:6] == ["small LVA_ERR_CAPACITY", "empty LVA_OK"]
    assert out[6:8] == ["prefix bytes 1", "rows -1"]
    assert out[8].startswith("append LVA_ERR_INVALID_ARG: append: lens_out")
    assert out[9].startswith("evict LVA_ERR_INVALID_ARG: evict: need 1 <= budget")
