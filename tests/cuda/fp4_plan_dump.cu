// Prints which kernel the 4-bit product takes, as the library chooses it, for shapes read
// from stdin ("M N K aligned sms" per line; aligned: the output is at a multiple of 16
// bytes): "pairs BN", BN weight rows to a tile, or "few BN KS", BN tokens to a tile and
// K split over KS CTAs, then 1 where a linear layer of the shape quantises inside the
// product. Host code only: no GPU is needed to run it.
#include <cstdio>

#include "gemm_fp4.cu"

namespace fp8blk {
int current_device(const DevInfo**) { return FP8BLK_ERR_CUDA; }
bool fp4_fmt_valid(int) { return true; }
int fp4_quant_launch(const void*, bool, int64_t, int64_t, int64_t, int, void*, void*, float*, int, bool, cudaStream_t) {
  return FP8BLK_ERR_CUDA;
}
}  // namespace fp8blk

int main() {
  long long M, N, K;
  int aligned, sms;
  while (std::scanf("%lld %lld %lld %d %d", &M, &N, &K, &aligned, &sms) == 5) {
    DevInfo d{};
    d.sm_count = sms;
    Fp4Params p{};
    p.M = M, p.N = N;
    p.c = reinterpret_cast<__nv_bfloat16*>(aligned ? 4096 : 4098);
    p.ktiles = K / 64;
    p.stages_k = static_cast<int>((K + kStageK - 1) / kStageK);
    p.tiles_n = static_cast<int>((N + 127) / 128);
    const int fused = fuses(&d, M, N, K);
    if (takes_pairs(&d, p) && pair_fits(p)) {
      std::printf("pairs %d %d\n", pair_columns(&d, p), fused);
    } else {
      const int bn = M <= 16 ? 16 : M <= 32 ? 32 : 64;
      std::printf("few %d %d %d\n", bn, few_split(p.tiles_n * ((M + bn - 1) / bn), p.stages_k, sms), fused);
    }
  }
  return 0;
}
