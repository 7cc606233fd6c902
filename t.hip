#include <hip/hip_runtime.h>
#include <stdint.h>
typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t v4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
__global__ void k(const uint16_t* p, uint16_t* q, float* f){
  int i = threadIdx.x;
  v4 a = *(const u4*)(p + i*8+1);
  __builtin_nontemporal_store((u4)a, (u4*)(q+i*8+1));
  f2 x = {f[i], f[i+1]};
  b2 r = __builtin_convertvector(x,b2);
  ((uint32_t*)f)[i+1000] = __builtin_bit_cast(uint32_t,r);
  f[i+3000] = __builtin_amdgcn_exp2f(x.x);
}
