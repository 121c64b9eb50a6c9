// Which kernel a dense product runs on: a rule on its sizes.
//
//  * Forward of up to 32 tokens (gated: 64): dense_few.cu.  1024 -> 4096: 6.0 us at 16 tokens,
//    where the pairs take 7.5; 8.1 at 64, where they take 7.2.  Gated, 768 -> 2048: 7.2 us at 64
//    tokens and 14.9 at 256, where the pairs take 8.7 and 8.9.
//  * Otherwise CTA pairs (dense_pair.cu) with the tile width and split that this estimate puts
//    lowest, in us.  A wave of tiles takes its K steps; a step takes `step` when a few pairs run
//    and `busy` when all do (they share the L2's bandwidth).  Persistent tiles overlap their
//    epilogues; split ones do not, and add the cluster's join.
//      weight gradient 768 x 768 over 32768 tokens: 43 us at 256 x 4 pairs, 97 at 128, 141 at 256
//      weight gradient 4096 x 1024 over 32768 tokens: 148 us at 256, 209 at 128, 173 at 256 x 2
//      input gradient 1024 <- 4096 of 1024 tokens: 12.1 us at 128 x 2, 14.6 at 128, 22.0 at 256
//      forward 768 -> 768 of 4096 tokens: 9.1 us at 256, 9.7 at 128, 19.4 at 256 x 2
//    It knows no epilogue, which costs either width about as much, so that the measured times lie
//    above it; with bias and residual, or activation and kept pre-activations:
//      forward 768 -> 768 of 8192 tokens, residual: 15.1 us at 256, 15.3 at 128 (without an epilogue
//      13.4 and 12.6; estimated 10.2 and 9.5, so 128 is taken: three rounds of 192 tiles)
//      forward 512 -> 2048 of 32768 tokens, gelu, kept: 63.9 us at 256, 70.9 at 128 (48.4 and 59.2)
#include "layer_ops.h"

namespace dfs {
namespace {

constexpr int64_t kFewTokens = 32, kFewTokensGated = 64;

struct Shape { int64_t I, J, K; };          // result rows and columns, summed length

double estimate(const Shape& s, int bn, bool gated, int splits) {
    const double step = bn == 256 ? 0.27 : 0.155, busy = bn == 256 ? 0.305 : 0.205;
    const int64_t width = gated ? bn / 2 : bn;
    const int64_t tiles = ((s.I + 255) / 256) * ((s.J + width - 1) / width);
    const int64_t steps = (s.K + 63) / 64, fit = dense_pair_clusters(splits);
    const int64_t waves = (tiles + fit - 1) / fit;
    const double load = tiles < fit ? (double)tiles / fit : 1.0;
    const double each = step + (busy - step) * load;
    if (splits == 1) return (bn == 256 ? 2.9 : 2.1) + (double)(waves * steps) * each;
    return (bn == 256 ? 5.2 : 3.6) + (double)(waves * ((steps + splits - 1) / splits)) * each + 6.0 * (double)(waves - 1);
}

struct Pick {
    int bn, splits;
    double us;
};

Shape shape_of(DenseForm form, const DenseArgs& a) {
    if (form == kForward) return {a.rows, a.gated ? a.cols / 2 : a.cols, a.inner};
    if (form == kInputGrad) return {a.rows, a.inner, a.cols};
    return {a.cols, a.inner, a.rows};
}

Pick pick(const Shape& s, bool gated) {
    Pick best{256, 1, estimate(s, 256, gated, 1)};
    for (int bn = 256; bn >= (gated ? 256 : 128); bn -= 128)
        for (int splits = 1; splits <= 4; splits *= 2) {
            if ((s.K + 63) / 64 < 2 * splits && splits > 1) continue;
            const double t = estimate(s, bn, gated, splits);
            if (t < best.us) best = {bn, splits, t};
        }
    return best;
}

}  // namespace

int launch_dense(DenseForm form, const DenseArgs& a, cudaStream_t stream) {
    if (form == kForward && a.rows <= (a.gated ? kFewTokensGated : kFewTokens)) return launch_dense_few(a, stream);
    const Pick p = pick(shape_of(form, a), form == kForward && a.gated);
    return launch_dense_pair(form, a, p.bn, p.splits, stream);
}

// Both gradients: one launch where its busiest pair ends before the two kernels after each
// other would (2 us for the second launch): 2.9 or 2.1 us and its K steps.
//   gated backward, 16384 x 1024 x 2816: 284 us in one launch, 318 in two (with the activations')
//   dense backward, 2048 x 1024 x 4096: 37 and 44;  1024 x 512 x 512: 12.2 and 17.7
//   dense backward, 32768 x 768 x 768, where the weights' gradient wants K split: 141 and 110
int launch_gradients(const DenseArgs& x, const DenseArgs& w, const BiasSums& bias, cudaStream_t stream) {
    const Pick px = pick(shape_of(kInputGrad, x), false), pw = pick(shape_of(kWeightGrad, w), false);
    const double at256 = 2.9 + 0.305 * (double)dense_grads_steps(x, 256);
    const double at128 = 2.1 + 0.205 * (double)dense_grads_steps(x, 128);
    if ((at256 < at128 ? at256 : at128) < px.us + pw.us + 2.0)
        return launch_dense_grads(x, w, bias, at256 <= at128 ? 256 : 128, stream);
    int st = bias.out ? launch_colsum(bias, stream) : DIFFUSER_OK;
    if (!st) st = launch_dense_pair(kInputGrad, x, px.bn, px.splits, stream);
    return st ? st : launch_dense_pair(kWeightGrad, w, pw.bn, pw.splits, stream);
}

}  // namespace dfs
