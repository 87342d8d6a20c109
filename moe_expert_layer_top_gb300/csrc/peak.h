// peak.h — the largest logit of a part of a row and the sum of its weights, and how two parts are joined.
//
// Lanes, warps and blocks join the same parts in butterflies, each pair with its own part first, and go on by what they
// get: all of them have to get the same bits. So the join must not depend on which side comes first. Written as
// sum * f + o.sum * g the compiler may round one product and not the other (a fused multiply-add); here each is rounded.
#pragma once

#include <cmath>

namespace moe {

// Largest logit (and the first token that has it), and the sum of 2^((x - top) c).
struct Peak {
  float top, sum;
  int token;

  // exp2: 2^x, 0 at -inf
  template <class Exp2>
  __device__ __forceinline__ void join(const Peak &o, float c, Exp2 exp2) {
    const float t = fmaxf(top, o.top), ref = t == -INFINITY ? 0.0f : t;
    sum = __fadd_rn(__fmul_rn(sum, exp2((top - ref) * c)), __fmul_rn(o.sum, exp2((o.top - ref) * c)));
    if (o.top > top || (o.top == top && o.token < token)) token = o.token;
    top = t;
  }
};

}  // namespace moe
