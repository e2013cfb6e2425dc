// linear_attention_tables.h -- what the tensor-core kernel of linear attention keeps in shared memory behind
// its tiles: tables of decays, scales and barriers.  Plain C++, so that its layout can be checked
// on the host.
#pragma once

#include <cstddef>
#include <cstdint>

namespace prnn {

struct Tables {
  float pw[132];              // l^n
  alignas(16) float dec[16];  // l^(15-j), or l^j in reverse; read four at a time
  // fp16: powers of two taken back from O2, U and O1, each kept until its last reader is sure to be done
  float x_scale[2], w_scale[4], row_scale[4][128];
  float red[2][8];
  float row_top[2][128];
  // l^(i-j) (in reverse l^(j-i)) of a 32 x 32 diagonal block, 0 where the mask is; read four at a time
  alignas(16) float diag[32][36];
  uint64_t ab_full[2], c_full[2], a_free[2], b_free[2], c_free[2], p_full[2], p_ready[2];
  uint64_t w_ready[2], o_full, o_free, o2_full, o2_free, x_ready, u_full, u_free, done;
  uint32_t tmem;
};
static_assert(offsetof(Tables, dec) % 16 == 0 && offsetof(Tables, diag) % 16 == 0 &&
                  sizeof(Tables::diag[0]) % 16 == 0 && alignof(Tables) == 16,
              "16-byte reads");
static_assert(offsetof(Tables, ab_full) % 8 == 0, "barriers");

}  // namespace prnn
