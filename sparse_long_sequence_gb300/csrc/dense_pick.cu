// Which kernel a dense product runs on: a rule on its sizes.
//
//  * Forward of up to 32 tokens: dense_few.cu.  (1024 -> 4096: 5.8 us at 16 tokens, where the
//    pairs take 7.1; 8.1 at 64 tokens, where they take 7.4.)
//  * Otherwise CTA pairs (dense_pair.cu) with the tile width and split that this estimate puts
//    lowest, in us.  A wave of tiles takes its K steps; a step takes `step` when a few pairs run
//    and `busy` when all do (they share the L2's bandwidth).  Persistent tiles overlap their
//    epilogues; split ones do not, and add the cluster's join.
//      weight gradient 768 x 768 over 32768 tokens: 44 us at 256 x 4 pairs, 98 at 128, 142 at 256
//      weight gradient 4096 x 1024 over 16384 tokens: 86 us at 256, 117 at 128, 170 at 256 x 2
//      input gradient 1024 <- 4096 of 1024 tokens: 12.3 us at 128 x 2, 15.1 at 128, 22.9 at 256
//      forward 768 -> 768 of 4096 tokens: 9.7 us at 256, 9.9 at 128, 19.6 at 256 x 2
#include "layer_ops.h"

namespace dfs {
namespace {

constexpr int64_t kFewTokens = 32;

struct Shape { int64_t I, J, K; };          // result rows and columns, summed length

double estimate(const Shape& s, int bn, bool gated, int splits) {
    const double step = bn == 256 ? 0.27 : 0.155, busy = bn == 256 ? 0.33 : 0.23;
    const int64_t width = gated ? bn / 2 : bn;
    const int64_t tiles = ((s.I + 255) / 256) * ((s.J + width - 1) / width);
    const int64_t steps = (s.K + 63) / 64, fit = dense_pair_clusters(splits);
    const int64_t waves = (tiles + fit - 1) / fit;
    const double load = tiles < fit ? (double)tiles / fit : 1.0;
    const double each = step + (busy - step) * load;
    if (splits == 1) return (bn == 256 ? 2.9 : 2.1) + (double)(waves * steps) * each;
    return (bn == 256 ? 5.2 : 3.6) + (double)(waves * ((steps + splits - 1) / splits)) * each + 6.0 * (double)(waves - 1);
}

}  // namespace

int launch_dense(DenseForm form, const DenseArgs& a, cudaStream_t stream) {
    const bool gated = form == kForward && a.gated;
    if (form == kForward && a.rows <= kFewTokens) return launch_dense_few(a, stream);
    Shape s;
    if (form == kForward) s = {a.rows, gated ? a.cols / 2 : a.cols, a.inner};
    else if (form == kInputGrad) s = {a.rows, a.inner, a.cols};
    else s = {a.cols, a.inner, a.rows};
    int best_bn = 256, best_splits = 1;
    double best = estimate(s, 256, gated, 1);
    for (int bn = 256; bn >= (gated ? 256 : 128); bn -= 128)
        for (int splits = 1; splits <= 4; splits *= 2) {
            if ((s.K + 63) / 64 < 2 * splits && splits > 1) continue;
            const double t = estimate(s, bn, gated, splits);
            if (t < best) { best = t; best_bn = bn; best_splits = splits; }
        }
    return launch_dense_pair(form, a, best_bn, best_splits, stream);
}

}  // namespace dfs
